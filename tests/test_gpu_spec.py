"""GPU parity of the speculative-decoding operations (quantised cache, tree
attention, verification, commit) against plain implementations in 64 bits."""
import ctypes
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

pytestmark = pytest.mark.gpu

DIMS = (32, 64, 128)


def dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
            "e4m3": torch.float8_e4m3fn}[name]


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def raw(t):
    """The bytes of a tensor on the host."""
    import torch
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---- the quantised cache ----------------------------------------------------------------

def e4m3_values():
    """The value of each of the 256 codes, from the format's definition."""
    out = []
    for code in range(256):
        sign, e, f = -1.0 if code & 128 else 1.0, code >> 3 & 15, code & 7
        v = math.ldexp(f / 8, -6) if e == 0 else math.ldexp(1 + f / 8, e - 7)
        out.append(math.nan if code & 127 == 127 else sign * v)
    return np.array(out)


E4M3 = e4m3_values()


def quantise64(x, kind):
    """Values and scales of float64 rows [..][D] by the definition in gpt2.h."""
    top = np.abs(x).max(-1)
    fine = np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        if kind == "int8":
            s = np.maximum(top.astype(np.float32) * (np.float32(1) / np.float32(127)),
                           np.float32(2.0 ** -126)).astype(np.float64)
            y = np.rint(np.where(fine[..., None], x, 0) / np.where(fine, s, 1)[..., None])
        else:
            e = np.array([max(-126, next(k for k in range(-200, 130) if t <= 448 * 2.0 ** k)) if f else 0
                          for t, f in zip(top.ravel(), fine.ravel())]).reshape(top.shape)
            s = 2.0 ** e
            z = np.where(fine[..., None], x, 0) / s[..., None]
            # nearest of the format's values; a tie goes to the even code
            order = np.array(sorted(range(127), key=lambda c: E4M3[c]))
            vals = E4M3[order]
            hi = np.clip(np.searchsorted(vals, np.abs(z)), 1, 126)
            lo = hi - 1
            dl, dh = np.abs(z) - vals[lo], vals[hi] - np.abs(z)
            pick = np.where((dl < dh) | ((dl == dh) & (order[lo] % 2 == 0)), lo, hi)
            y = np.sign(z) * vals[pick]
    return y, np.where(fine, s, np.nan)


def rows_with_edges(rng, n, H, D, src):
    """Random rows, and rows of zeros, subnormals, huge values, exact ties, an
    infinity, a NaN and a single value, as the source type holds them."""
    import torch
    x = rng.standard_normal((n, H, D)) * np.exp(rng.standard_normal((n, H, 1)))
    edges = [np.zeros(D), np.full(D, 1e-41), np.where(np.arange(D) % 2, 3.0e38, -1.5e38),
             np.r_[127.0, np.arange(1, D) - 20.5] * 0.25, np.r_[np.inf, np.ones(D - 1)], np.r_[1.0, np.nan, np.ones(D - 2)],
             np.r_[np.zeros(D - 1), 5e-3], np.r_[448.0, (np.arange(1, D) % 16 + 16.5) * 2.0 ** (np.arange(1, D) % 5 - 3)],
             np.r_[449.0, np.ones(D - 1)], np.full(D, 2.0 ** -126 * 100)]
    for i, e in enumerate(edges):
        if i < n:
            x[i, i % H] = e
    return torch.from_numpy(x.astype(np.float32)).to(dt(src)).cuda()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["int8", "e4m3", "f32", "f16", "bf16"])
def test_store_writes_the_definition(src, cache, D):
    """Codes and scales are exactly those of the definition (rounding of the
    exact quotient), the other rows of the cache stay as they were, rows
    outside it are skipped; the source lies inside wider rows, once aligned
    and once one element off."""
    import torch
    rng = np.random.default_rng(D)
    n, H, S, P = 37, 3, 4, 19
    x, y = rows_with_edges(rng, n, H, D, src), rows_with_edges(rng, n, H, D, src).flip(0)
    where = rng.permutation(S * P)[:n]
    slot, pos = where // P, where % P
    slot[n - 4:] = [-1, S, 1, 2]
    pos[n - 4:] = [0, 0, -1, P]
    for shift in (0, 1):
        wide = torch.zeros((n, 2 * H * D + 8 + shift), dtype=x.dtype, device="cuda")
        k = wide[:, shift:shift + H * D].unflatten(1, (H, D))
        v = wide[:, shift + H * D:shift + 2 * H * D].unflatten(1, (H, D))
        k.copy_(x)
        v.copy_(y)
        kc = torch.full((S, H, P, D), 3.0, device="cuda").to(dt(cache))
        vc = torch.full((S, H, P, D), 5.0, device="cuda").to(dt(cache))
        scaled = cache in ("int8", "e4m3")
        ks, vs = (torch.full((S, H, P), 7.0, device="cuda") for _ in range(2)) if scaled else (None, None)
        binding.op_kv_store(k, v, kc, vc, i32(slot), i32(pos), ks, vs)
        for src_rows, c, sc, fill in ((x, kc, ks, 3.0), (y, vc, vs, 5.0)):
            r = src_rows.float().cpu().numpy().astype(np.float64)
            want = torch.full((S, H, P, D), fill).to(dt(cache)).float().numpy().astype(np.float64)
            want_s = np.full((S, H, P), 7.0)
            if scaled:
                val, s = quantise64(r, cache)
            else:
                val, s = src_rows.float().cpu().to(dt(cache)).float().numpy().astype(np.float64), None
            for i in range(n):
                if 0 <= slot[i] < S and 0 <= pos[i] < P:
                    want[slot[i], :, pos[i]] = val[i]
                    if scaled:
                        want_s[slot[i], :, pos[i]] = s[i]
            got = c.cpu().float().numpy().astype(np.float64)
            assert np.array_equal(got, want, equal_nan=True)
            if scaled:
                assert np.array_equal(sc.cpu().numpy().astype(np.float64), want_s, equal_nan=True)


@pytest.mark.parametrize("cache", ["int8", "e4m3", "f32", "f16", "bf16"])
@pytest.mark.parametrize("dst", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
def test_load_reads_back(cache, dst, D):
    """Widened values, or code * scale rounded to fp32 and then to the row
    type; the same cache row twice, rows outside the cache as zeros, rows
    written into wider ones."""
    import torch
    rng = np.random.default_rng(D + 1)
    S, H, P, n = 3, 5, 11, 50
    kc = torch.from_numpy(rng.standard_normal((S, H, P, D)).astype(np.float32) * 60).to(dt(cache)).cuda()
    vc = torch.from_numpy(rng.standard_normal((S, H, P, D)).astype(np.float32) * 60).to(dt(cache)).cuda()
    scaled = cache in ("int8", "e4m3")
    ks, vs = (torch.from_numpy(np.exp(rng.standard_normal((S, H, P))).astype(np.float32)).cuda()
              for _ in range(2)) if scaled else (None, None)
    slot, pos = rng.integers(0, S, n), rng.integers(0, P, n)
    slot[:3], pos[3] = [-1, S, 1 << 30], -5
    out = torch.full((n, 2 * H * D + 3), 9.0, dtype=dt(dst), device="cuda")
    k, v = (out[:, a * H * D + a:(a + 1) * H * D + a].unflatten(1, (H, D)) for a in (0, 1))
    binding.op_kv_load(kc, vc, i32(slot), i32(pos), ks, vs, k=k, v=v)
    k2, v2 = binding.op_kv_load(kc, vc, i32(slot), i32(pos), ks, vs, dtype=dt(dst))
    for got, got2, c, sc in ((k, k2, kc, ks), (v, v2, vc, vs)):
        x = c.cpu().float()
        if scaled:
            x = x * sc.cpu().unsqueeze(-1)
        want = torch.zeros((n, H, D))
        for i in range(4, n):
            want[i] = x[slot[i], :, pos[i]]
        want = want.to(dt(dst))
        assert torch.equal(got.cpu(), want) and torch.equal(got2.cpu(), want)
    assert (out[:, H * D] == 9).all() and (out[:, 2 * H * D + 1:] == 9).all()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["int8", "e4m3", "f32", "f16", "bf16"])
def test_prompts_through_the_cache(src, cache, D):
    """Prompt-sized calls (several rows per thread; a last block that is not
    full): the codes and scales of 13,003 rows against the definition in 64 bits
    on the GPU, and the same rows read back as each row type."""
    import torch
    n, H, S, P = 13003, 5, 40, 400
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    x, y = ((torch.randn((n, H, D), generator=g, device="cuda") *
             torch.exp(torch.randn((n, H, 1), generator=g, device="cuda"))).to(dt(src)) for _ in range(2))
    at = torch.randperm(S * P, generator=g, device="cuda")[:n]
    slot, pos = (at // P).int(), (at % P).int()
    kc, vc = (torch.zeros((S, H, P, D), device="cuda").to(dt(cache)) for _ in range(2))
    scaled = cache in ("int8", "e4m3")
    ks, vs = (torch.zeros((S, H, P), device="cuda") for _ in range(2)) if scaled else (None, None)
    binding.op_kv_store(x, y, kc, vc, slot, pos, ks, vs)
    for rows, c, sc in ((x, kc, ks), (y, vc, vs)):
        d = rows.double()
        if cache == "int8":
            want_s = (rows.float().abs().amax(-1) * torch.full((), 1.0 / 127, device="cuda")).clamp(min=2.0 ** -126)
            want = torch.round(d / want_s.double().unsqueeze(-1))
        elif cache == "e4m3":
            m, e = torch.frexp(d.abs().amax(-1) / 448)      # (exact; a logarithm is not, at a power of two)
            want_s = torch.exp2(torch.where(m == 0.5, e - 1, e).clamp(min=-126).float())
            want = (d / want_s.double().unsqueeze(-1)).float().to(torch.float8_e4m3fn).double()
        else:
            want, want_s = rows.to(dt(cache)).double(), None
        got = c[slot.long(), :, pos.long()] if cache != "e4m3" else \
            c.view(torch.uint8)[slot.long(), :, pos.long()].view(c.dtype)
        assert torch.equal(got.double(), want)
        if scaled:
            assert torch.equal(sc[slot.long(), :, pos.long()], want_s)
    for dst in ("f32", "f16", "bf16"):
        k, v = binding.op_kv_load(kc, vc, slot, pos, ks, vs, dtype=dt(dst))
        for got, c, sc in ((k, kc, ks), (v, vc, vs)):
            w = c.view(torch.uint8)[slot.long(), :, pos.long()].view(c.dtype).float() if cache == "e4m3" else \
                c[slot.long(), :, pos.long()].float()
            if scaled:
                w = w * sc[slot.long(), :, pos.long()].unsqueeze(-1)
            assert torch.equal(got, w.to(dt(dst)))


# ---- tree attention ---------------------------------------------------------------------

COMBOS = [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("f32", "int8"), ("f32", "e4m3"), ("bf16", "bf16"),
          ("f16", "f16"), ("bf16", "int8"), ("f16", "int8"), ("bf16", "e4m3"), ("f16", "e4m3")]


def random_tree(rng, n, width=3):
    return [-1] + [int(rng.integers(max(0, i - width), i)) for i in range(1, n)]


def make_cache(rng, kind, S, K, P, D):
    import torch
    x = torch.from_numpy(rng.standard_normal((S, K, P, D)).astype(np.float32))
    if kind == "int8":
        return ((x * 40).round().clamp(-127, 127).to(torch.int8).cuda(),
                torch.from_numpy((0.02 * np.exp(rng.standard_normal((S, K, P)))).astype(np.float32)).cuda())
    if kind == "e4m3":
        return ((x * 60).clamp(-448, 448).to(torch.float8_e4m3fn).cuda(),
                torch.from_numpy((2.0 ** rng.integers(-8, -3, (S, K, P))).astype(np.float32)).cuda())
    return x.to(dt(kind)).cuda(), None


def attend64(q, kc, vc, ks, vs, slot, cached, first, mask, scale):
    """Per (sequence, head, node) in float64, and the error allowed for each
    element (see check_attention)."""
    import torch
    q = q.float().cpu().numpy().astype(np.float64)
    n, H, D = q.shape
    S, K, P, _ = kc.shape

    def wide(c, s):
        c = c.cpu().float().numpy().astype(np.float64)
        return c if s is None else c * s.cpu().numpy().astype(np.float64)[..., None]

    k, v = wide(kc, ks), wide(vc, vs)
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    for b in range(len(slot)):
        if not 0 <= slot[b] < S:
            continue
        c = min(max(cached[b], 0), P)
        for t in range(first[b + 1] - first[b]):
            r = first[b] + t
            m = int(mask[r]) & (2 ** 64 - 1)
            see = list(range(c)) + [c + j for j in range(first[b + 1] - first[b]) if m >> j & 1 and c + j < P]
            if not see:
                continue
            for h in range(H):
                kk, vv = k[slot[b], h // (H // K)][see], v[slot[b], h // (H // K)][see]
                a = kk @ q[r, h] * scale
                w = np.exp(a - a.max())
                w /= w.sum()
                out[r, h] = w @ vv
                size = (np.abs(kk) @ np.abs(q[r, h])).max() * abs(scale)
                tol[r, h] = (2 * size * 2.0 ** -18 + 2.0 ** -16) * (w @ np.abs(vv))
                if kc.dtype not in (torch.float32, torch.bfloat16):
                    # weights enter as two fp16 parts in units of 2^-13 of the largest
                    # (of the largest value scale too, rounded up to a power of two,
                    # where values have scales): what the second part drops below
                    # fp16's smallest step, 2^-24, is at most half of it, 2^-25 /
                    # 2^13 of the largest value per row of the cache that is seen
                    unit = 1.0 if vs is None else 2 * float(np.nanmax(vs.cpu().numpy()[slot[b], h // (H // K), see]))
                    code = vc[slot[b], h // (H // K)].float().abs()
                    tol[r, h] += len(see) * 2.0 ** -38 * unit * float(code[see].max())
    return out, tol


def check_attention(got, want, tol):
    """The products keep at least 21 bits of q, k and v and 16 of the weights,
    and sum at most 128 / 8 + 8 partial sums in fp32 (each off by at most
    2^-23): a score is off by less than 2^-18 of sum |q k| scale, a weight by
    that much relatively, twice (numerator and denominator), plus 2^-16 for
    its own parts and the sums; then half a step of the result's type."""
    import torch
    g = got.double().cpu().numpy()
    lim = tol + np.abs(want) * torch.finfo(got.dtype).eps / 2 + 1e-30
    if got.dtype == torch.float16:
        lim = lim + 2.0 ** -25           # half a step below fp16's normal numbers
    err = np.abs(g - want)
    assert np.all(err <= lim), f"worst {np.nanmax(err / lim):.3g} of what is allowed, {err.max():.3g}"


def run_attention(rng, qt, ct, D, K, G, P, cached, counts, slots=None, scale=None, masks=None, extra=0, S=None):
    import torch
    B = len(cached)
    S = S or B + 1
    kc, ks = make_cache(rng, ct, S, K, P, D)
    vc, vs = make_cache(rng, ct, S, K, P, D)
    slot = rng.permutation(S)[:B] if slots is None else slots
    first = np.concatenate([[0], np.cumsum(counts)])
    if masks is None:
        masks = np.concatenate([binding.tree_masks(random_tree(rng, c)) if c else np.zeros(0, np.int64)
                                for c in counts])
    n = int(first[-1]) + extra
    masks = np.concatenate([masks, np.full(extra, -1, np.int64)])
    q = torch.from_numpy((1.5 * rng.standard_normal((n, K * G, D))).astype(np.float32)).to(dt(qt)).cuda()
    scale_ = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full_like(q, 77.0)
    got = binding.op_tree_attention(q, kc, vc, i32(slot), i32(cached), i32(first), torch.from_numpy(masks).cuda(),
                                    max(1, max(counts)), ks, vs, scale=scale, out=out)
    assert got is out
    want, tol = attend64(q, kc, vc, ks, vs, slot, cached, first, masks, scale_)
    f = int(first[-1])
    check_attention(got[:f], want[:f], tol[:f])
    assert (got[f:] == 77).all()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("qt,ct", COMBOS)
def test_tree_attention_types(qt, ct, D):
    """Every type and head size: ragged prefixes around the tile sizes, trees
    of up to 16 nodes, a sequence without nodes, one without a prefix, rows
    behind the last sequence."""
    rng = np.random.default_rng(D)
    run_attention(rng, qt, ct, D, 2, 1, 301, [0, 31, 33, 100, 285, 64], [5, 16, 1, 0, 16, 7], extra=3)


@pytest.mark.parametrize("qt,ct", [("f32", "f32"), ("f32", "bf16"), ("f32", "int8"), ("bf16", "bf16"), ("f16", "f16"),
                                   ("bf16", "int8"), ("f16", "e4m3")])
@pytest.mark.parametrize("counts,G,D", [([64, 33, 17], 1, 64), ([20, 3], 3, 64), ([40, 1], 1, 128), ([9], 8, 128),
                                        ([64], 2, 32), ([32, 16], 1, 32)])
def test_tree_attention_many_rows(qt, ct, counts, G, D):
    """More than 16 rows of a (sequence, cache head): two row tiles in a warp,
    several row tiles, grouped heads."""
    rng = np.random.default_rng(sum(counts) + G)
    run_attention(rng, qt, ct, D, 2, G, 500, [int(x) for x in rng.integers(0, 430, len(counts))], counts)


@pytest.mark.parametrize("counts,G,D", [([64, 33, 17], 1, 64), ([20, 3], 3, 64), ([40, 1], 1, 128), ([9], 8, 128),
                                        ([17], 1, 128), ([21, 0, 32], 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tree_attention_many_rows_long_caches(dtype, counts, G, D):
    """The same over caches of many positions (of which few are used), where the
    tensor cores' kernel takes over: fewer tiles than SMs, parts of units."""
    rng = np.random.default_rng(sum(counts) + G + D)
    cached = [int(x) for x in rng.integers(0, 3000, len(counts))]
    run_attention(rng, dtype, dtype, D, 2, G, 36000 // len(counts), cached, counts)


@pytest.mark.parametrize("counts,G", [([64, 33, 17], 1), ([20, 3], 3), ([40, 1], 1), ([9], 4), ([17], 1), ([21, 0, 32], 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tree_attention_many_rows_longest_caches(dtype, counts, G):
    """64 dimensions in caches so long that the tensor cores' kernel takes over
    for few sequences too."""
    rng = np.random.default_rng(sum(counts) + G)
    cached = [int(x) for x in rng.integers(0, 3000, len(counts))]
    run_attention(rng, dtype, dtype, 64, 2, G, 130000 // len(counts), cached, counts, S=len(counts))


@pytest.mark.parametrize("counts,G,D", [(17, 1, 64), (33, 1, 128), (5, 4, 128), (40, 2, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tree_attention_many_units(dtype, counts, G, D):
    """Many more (sequence, cache head, row tile) units than SMs, of ragged
    lengths from no cached row to several tiles: a CTA works through several
    units, and units are shared between CTAs."""
    rng = np.random.default_rng(counts + D)
    B, K = 30, 9
    cached = [int(x) for x in rng.integers(0, 700, B)]
    cached[3] = cached[17] = 0
    n = [int(x) for x in rng.integers(1, counts + 1, B)]
    n[0], n[5], n[20] = counts, 0, 0
    run_attention(rng, dtype, dtype, D, K, G, 1600, cached, n)


@pytest.mark.parametrize("qt,ct", COMBOS)
def test_single_tokens_long_and_short(qt, ct):
    """The decode form (one node per sequence), from no cached row to long
    caches split over a cluster."""
    rng = np.random.default_rng(5)
    run_attention(rng, qt, ct, 64, 1, 1, 5003, [0, 1, 2, 15, 16, 17, 4999, 5002], [1] * 8)
    run_attention(rng, qt, ct, 128, 1, 4, 3001, [2900], [1])


@pytest.mark.parametrize("qt,ct", COMBOS)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("P,K", [(700, 2), (2600, 3), (300, 30)])
def test_few_rows(qt, ct, D, P, K):
    """One to eight query rows per cache head, nodes and heads of a group, with
    little and much beside them: tiles of one, two, four and sixteen rows, odd
    rests, several CTAs per cache."""
    rng = np.random.default_rng(P + D)
    for G, counts in ((1, [1, 1]), (2, [1]), (1, [2, 1, 0]), (1, [3]), (4, [1, 1]), (1, [5, 2]), (7, [1]), (2, [4, 3])):
        cached = [int(x) for x in rng.integers(0, P, len(counts))]
        run_attention(rng, qt, ct, D, K, G, P, cached, counts, extra=1)


@pytest.mark.parametrize("P", [1, 2, 31, 77, 128])
@pytest.mark.parametrize("ct", ["f32", "int8"])
def test_small_caches(P, ct):
    """Caches of one position and odd sizes, filled to the end; nodes whose row
    would lie outside are not seen."""
    rng = np.random.default_rng(P)
    run_attention(rng, "f32", ct, 32, 3, 1, P, [0, P, P - 1, max(0, P - 3)], [1, 1, 1, min(P, 5)])
    run_attention(rng, "f32", ct, 32, 1, 1, P, [P, P + 5, max(0, P - 2)], [4, 3, 6])


def test_masks_decide():
    """Any mask: nothing at all (zeros with no prefix), single nodes, all 64
    nodes; a slot outside the cache gives zeros."""
    import torch
    rng = np.random.default_rng(8)
    masks = rng.integers(-2 ** 63, 2 ** 63 - 1, 64 + 9)
    masks[[0, 3, 64, 66]] = 0
    masks[5] = -1
    run_attention(rng, "bf16", "bf16", 64, 2, 1, 200, [0, 50], [64, 9], masks=masks)
    run_attention(rng, "f32", "f32", 64, 2, 1, 200, [0, 50], [64, 9], masks=masks, slots=np.array([2, -1]))
    run_attention(rng, "f32", "f32", 64, 2, 1, 90, [-7, 50], [3, 2], masks=np.array([1, 0, 6, 0, 2]))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    rng = np.random.default_rng(9)
    run_attention(rng, "f32", "f16", 64, 2, 1, 120, [90, 11], [6, 2], scale=scale)


@pytest.mark.parametrize("qt,ct", COMBOS)
def test_what_is_not_seen_does_not_enter(qt, ct):
    """Infinities and NaN in cache rows behind the nodes, in other nodes' keys,
    values and scales: nodes that do not see them are as without them, nodes
    that do are not finite."""
    import torch
    rng = np.random.default_rng(11)
    K, D, P, c, n = 2, 64, 150, 60, 9
    kc, ks = make_cache(rng, ct, 1, K, P, D)
    vc, vs = make_cache(rng, ct, 1, K, P, D)
    parents = [-1, 0, 0, 1, 2, 3, 4, 5, 6]
    mask = binding.tree_masks(parents)
    q = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).to(dt(qt)).cuda()
    args = (i32([0]), i32([c]), i32([0, n]), torch.from_numpy(mask).cuda(), n)
    want, tol = attend64(q, kc, vc, ks, vs, [0], [c], [0, n], mask, 1 / 8)
    stale = torch.full((1, K, P - c - n, D), math.nan, device="cuda")
    if ct == "int8":
        ks[:, :, c + n:], vs[:, :, c + n:] = math.nan, math.inf
    else:
        kc[:, :, c + n:] = stale.to(kc.dtype)
        vc[:, :, c + n:] = (stale if ct == "e4m3" else stale + math.inf).to(kc.dtype)
    check_attention(binding.op_tree_attention(q, kc, vc, *args, ks, vs), want, tol)
    # node 4 (seen by 4, 6 and 8) is poisoned in one place after another
    sees = np.array([(int(m) >> 4) & 1 for m in mask], bool)
    spots = []
    if ks is not None:
        spots += [(ks, (0, 1, c + 4), math.nan), (vs, (0, 1, c + 4), math.nan), (vs, (0, 1, c + 4), math.inf)]
    if ct != "int8":
        bad = [math.nan] if ct == "e4m3" else [math.nan, math.inf, -math.inf]
        spots += [(t, (0, 1, c + 4, 17), x) for t in (kc, vc) for x in bad]
    for t, at, x in spots:
        old = t[at].clone()
        t[at] = torch.tensor(x).to(t.dtype)
        got = binding.op_tree_attention(q, kc, vc, *args, ks, vs)
        t[at] = old
        check_attention(got[~sees], want[~sees], tol[~sees])
        check_attention(got[:, 0], want[:, 0], tol[:, 0])
        whole = t is ks or t is vs or t is kc
        if t is kc and not math.isnan(x):
            continue                     # (a score of -infinity has weight zero: a finite result is right)
        hit = got[sees][:, 1] if whole else got[sees][:, 1, 17]
        assert not torch.isfinite(hit.float()).any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("c,n,K,P", [(60, 24, 200, 1600), (1500, 24, 2, 40000), (1020, 40, 1, 70000),
                                     (60, 24, 3, 200)])
def test_what_is_not_seen_does_not_enter_many_rows(dtype, D, c, n, K, P):
    """The same with more than 16 query rows: units within one CTA's share
    (200 heads of one tile), units that many CTAs share, and a short cache."""
    import torch
    rng = np.random.default_rng(c + n)
    kc, _ = make_cache(rng, dtype, 1, K, P, D)
    vc, _ = make_cache(rng, dtype, 1, K, P, D)
    mask = binding.tree_masks(random_tree(rng, n, 6))
    q = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).to(dt(dtype)).cuda()
    args = (i32([0]), i32([c]), i32([0, n]), torch.from_numpy(mask).cuda(), n)
    h = K - 1                                     # (heads alike: the reference for the poisoned one)
    want, tol = attend64(q[:, h:], kc[:, h:], vc[:, h:], None, None, [0], [c], [0, n], mask, 1 / math.sqrt(D))
    kc[:, :, c + n:] = math.nan
    vc[:, :, c + n:] = math.inf
    base = binding.op_tree_attention(q, kc, vc, *args)
    check_attention(base[:, h:], want, tol)
    node = 4
    sees = np.array([(int(m) >> node) & 1 for m in mask], bool)
    assert sees.any() and not sees.all()
    for t, x in [(vc, math.nan), (vc, math.inf), (vc, -math.inf), (kc, math.nan)]:
        at = (0, h, c + node, 17)
        old = t[at].clone()
        t[at] = x
        got = binding.op_tree_attention(q, kc, vc, *args)
        t[at] = old
        assert torch.equal(got[:, :h], base[:, :h])
        check_attention(got[~sees][:, h:], want[~sees], tol[~sees])
        hit = got[sees][:, h] if t is kc else got[sees][:, h, 17]
        assert not torch.isfinite(hit.float()).any()
        if t is vc:
            rest = [d for d in range(D) if d != 17]
            check_attention(got[sees][:, h:][..., rest], want[sees][..., rest], tol[sees][..., rest])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("c,n,K,P", [(1500, 24, 2, 130000), (1020, 40, 1, 180000)])
def test_what_is_not_seen_does_not_enter_longest_caches(dtype, c, n, K, P):
    test_what_is_not_seen_does_not_enter_many_rows(dtype, 64, c, n, K, P)


def test_wide_value_scales():
    """int8 value scales that differ by 2^40 within a sequence, rising and
    falling over the tiles, zero among them."""
    import torch
    rng = np.random.default_rng(12)
    K, D, P, c = 1, 64, 400, 390
    kc, ks = make_cache(rng, "int8", 1, K, P, D)
    vc, vs = make_cache(rng, "int8", 1, K, P, D)
    vs.copy_(torch.from_numpy(2.0 ** rng.integers(-20, 21, (1, K, P))).float())
    vs[0, 0, ::7] = 0
    q = torch.from_numpy(rng.standard_normal((2, K, D)).astype(np.float32)).cuda()
    mask = binding.tree_masks([-1, 0])
    got = binding.op_tree_attention(q, kc, vc, i32([0]), i32([c]), i32([0, 2]), torch.from_numpy(mask).cuda(), 2, ks, vs)
    want, tol = attend64(q, kc, vc, ks, vs, [0], [c], [0, 2], mask, 1 / 8)
    check_attention(got, want, tol)


def test_large_and_small_queries():
    """Rows of very different size (the powers of two that bring q into fp16's
    range are per row): 2^-60 to 2^12."""
    import torch
    rng = np.random.default_rng(13)
    K, D, P, n = 2, 64, 100, 12
    for ct in ("int8", "f16", "bf16", "f32"):
        kc, ks = make_cache(rng, ct, 1, K, P, D)
        vc, vs = make_cache(rng, ct, 1, K, P, D)
        size = 2.0 ** np.array([-60, -40, -20, -10, -5, 0, 1, 2, 3, 4, 5, -126])
        q = torch.from_numpy((rng.standard_normal((n, K, D)) * size[:, None, None]).astype(np.float32)).cuda()
        q[3] = 0
        mask = binding.tree_masks(list(range(-1, n - 1)))
        got = binding.op_tree_attention(q, kc, vc, i32([0]), i32([70]), i32([0, n]), torch.from_numpy(mask).cuda(), n,
                                        ks, vs)
        want, tol = attend64(q, kc, vc, ks, vs, [0], [70], [0, n], mask, 1 / 8)
        check_attention(got, want, tol)


def test_strided_rows_streams_and_graphs():
    """q inside fused QKV rows and out inside wider rows; the same bits on
    another stream, twice in flight on two streams, and from a captured
    graph replayed on new inputs."""
    import torch
    rng = np.random.default_rng(14)
    K, D, P, counts, cached = 3, 64, 260, [8, 5], [200, 33]
    kc, ks = make_cache(rng, "int8", 2, K, P, D)
    vc, vs = make_cache(rng, "int8", 2, K, P, D)
    mask = np.concatenate([binding.tree_masks(random_tree(rng, c)) for c in counts])
    first, n, E = [0, 8, 13], 13, K * D
    qkv = torch.from_numpy(rng.standard_normal((n, 3 * E)).astype(np.float32)).cuda()
    q = qkv[:, :E].unflatten(1, (K, D))
    args = (i32([1, 0]), i32(cached), i32(first), torch.from_numpy(mask).cuda(), 8, ks, vs)
    want, tol = attend64(q, kc, vc, ks, vs, [1, 0], cached, first, mask, 1 / 8)
    base = binding.op_tree_attention(q, kc, vc, *args)
    check_attention(base, want, tol)
    wide = torch.full((n, 2 * E), 4.0, device="cuda")
    out = binding.op_tree_attention(q, kc, vc, *args, out=wide[:, E:].unflatten(1, (K, D)))
    assert torch.equal(out, base) and (wide[:, :E] == 4).all()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [binding.op_tree_attention(q, kc, vc, *args, stream=s) for s in (s1, s2, s1)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, base) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = binding.op_tree_attention(q, kc, vc, *args)
    qkv.mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    want2, tol2 = attend64(q, kc, vc, ks, vs, [1, 0], cached, first, mask, 1 / 8)
    check_attention(held, want2, tol2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_ragged_batches(dtype, D):
    """The tensor cores' kernel on a batch with slots outside the cache, two
    sequences of one slot, sequences without nodes or cached rows, lengths past
    the cache's end and negative ones, nodes behind max_nodes (left as they
    were) and rows behind the last sequence."""
    import torch
    rng = np.random.default_rng(17)
    K, P, S, mx = 5, 1700, 40, 24
    cached = [int(x) for x in rng.integers(0, 900, 30)]
    cached[:6] = [P - 5, P, P + 9, -3, 0, 1]
    counts = [int(x) for x in rng.integers(1, mx + 1, 30)]
    counts[:9] = [24, 24, 24, 24, 24, 0, 24, 24, 40]     # (one of more than max_nodes)
    slot = [int(x) for x in rng.permutation(S)[:30]]
    slot[6], slot[7], slot[9] = -1, S, slot[10]
    first = np.concatenate([[0], np.cumsum(counts)])
    masks = np.concatenate([binding.tree_masks(random_tree(rng, c)) if c else np.zeros(0, np.int64) for c in counts])
    n = int(first[-1]) + 3
    masks = np.concatenate([masks, np.full(3, -1, np.int64)])
    masks[first[12]] = 0                                 # a node that sees the prefix only
    masks[first[4] + 1] = 0                              # ... and one that sees nothing
    kc, vc = (make_cache(rng, dtype, S, K, P, D)[0] for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).to(dt(dtype)).cuda()
    out = torch.full_like(q, 77.0)
    binding.op_tree_attention(q, kc, vc, i32(slot), i32(cached), i32(first), torch.from_numpy(masks).cuda(), mx, out=out)
    seen = masks.copy()                                  # (no cache rows beyond max_nodes nodes)
    seen[first[8]:first[9]] &= (1 << mx) - 1
    want, tol = attend64(q, kc, vc, None, None, slot, cached, first, seen, 1 / math.sqrt(D))
    kept = np.ones(n, bool)
    kept[first[8] + mx:first[9]] = False
    kept[first[-1]:] = False
    k = torch.from_numpy(kept).cuda()
    assert (out[~k] == 77).all()
    check_attention(out[k], want[kept], tol[kept])
    assert (out[first[4] + 1] == 0).all() and (out[first[6]:first[8]] == 0).all()


def test_many_rows_more_sequences_than_threads():
    """700 sequences over three slots: the list of tiles is searched in steps."""
    rng = np.random.default_rng(18)
    B = 700
    counts = [int(x) for x in rng.integers(0, 4, B)]
    counts[0], counts[699] = 17, 9
    run_attention(rng, "bf16", "bf16", 64, 1, 1, 1536, [int(x) for x in rng.integers(0, 200, B)], counts,
                  slots=[int(x) for x in rng.integers(0, 3, B)], S=3)


@pytest.mark.parametrize("counts,D,P", [([24, 40, 3], 64, 8000), ([24, 40, 3], 64, 16000), ([64, 2], 128, 8000)])
def test_many_rows_strided_streams_and_graphs(counts, D, P):
    """The tensor cores' kernel: q inside fused rows, out inside wider ones; the
    same bits on another stream, with two calls in flight, with a workspace of
    the caller's, and from two captured graphs that share it."""
    import torch
    rng = np.random.default_rng(19)
    B, K = len(counts), 4
    cached = [int(x) for x in rng.integers(0, 1500, B)]
    kc, vc = (make_cache(rng, "bf16", B, K, P, D)[0] for _ in range(2))
    masks = np.concatenate([binding.tree_masks(random_tree(rng, c)) for c in counts])
    first = np.concatenate([[0], np.cumsum(counts)])
    n, E = int(first[-1]), K * D
    qkv = torch.from_numpy(rng.standard_normal((n, 3 * E)).astype(np.float32)).bfloat16().cuda()
    q = qkv[:, E:2 * E].unflatten(1, (K, D))
    args = (i32(np.arange(B)), i32(cached), i32(first), torch.from_numpy(masks).cuda(), max(counts))
    base = binding.op_tree_attention(q, kc, vc, *args)
    want, tol = attend64(q, kc, vc, None, None, list(range(B)), cached, first, masks, 1 / math.sqrt(D))
    check_attention(base, want, tol)
    wide = torch.full((n, 2 * E), 4.0, device="cuda", dtype=torch.bfloat16)
    out = binding.op_tree_attention(q, kc, vc, *args, out=wide[:, E:].unflatten(1, (K, D)))
    assert torch.equal(out, base) and (wide[:, :E] == 4).all()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [binding.op_tree_attention(q, kc, vc, *args, stream=s) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, base) for o in outs)
    kv = binding.KV(kc.data_ptr(), vc.data_ptr(), None, None, binding.GPT2_BF16, B, K, P, D)
    need = binding.lib().gpt2_op_tree_attention_workspace(ctypes.byref(kv), binding.GPT2_BF16, K, max(counts))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for bad in (ws[:need - 16], ws[16:], torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(binding.GPT2Error):
            binding.op_tree_attention(q, kc, vc, *args, workspace=bad)
    graphs, held, q2 = [], [], (-0.5 * q).contiguous()
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(binding.op_tree_attention(x, kc, vc, *args, workspace=ws))
        graphs.append(g)
    for k in (0, 1, 0, 1, 1):
        held[k].zero_()
        graphs[k].replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], base) and torch.equal(held[1], binding.op_tree_attention(q2, kc, vc, *args))


def test_chained_calls_and_joined_streams():
    """Calls that feed one another, back to back (each may be placed before the
    last one has ended), and in a captured graph whose branches fork and join
    between them; many times, with inputs that an ordinary operation writes just
    before."""
    import torch
    rng = np.random.default_rng(20)
    B, K, P, D, n = 6, 4, 2100, 64, 8
    kc, vc = (torch.zeros((2, B, K, P, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((2, B, K, P), device="cuda") for _ in range(2))
    cached = i32(rng.integers(0, 1500, B))
    first, slot = i32(np.arange(B + 1) * n), i32(rng.permutation(B))
    mask = torch.from_numpy(np.tile(binding.tree_masks(random_tree(rng, n)), B)).cuda()
    rs, rp = slot.repeat_interleave(n), (cached.repeat_interleave(n) + torch.arange(n, device="cuda").repeat(B)).int()
    src = torch.from_numpy(rng.standard_normal((3, B * n, K, D)).astype(np.float32)).cuda()
    x = torch.empty_like(src)
    path = i32([[0, 2, 3, -1, -1, -1, -1, -1]] * B)
    n_path = i32([3] * B)
    side = torch.cuda.Stream()

    def chain(fork):
        outs = []
        torch.mul(src, 1.0, out=x)
        for layer in range(2):
            c = (kc[layer], vc[layer])
            binding.op_kv_store(x[1], x[2], *c, rs, rp, ks[layer], vs[layer])
            if fork:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    outs.append(binding.op_kv_load(*c, rs, rp, ks[layer], vs[layer])[0])
            outs.append(binding.op_tree_attention(x[0], *c, slot, cached, first, mask, n, ks[layer], vs[layer]))
            if fork:
                torch.cuda.current_stream().wait_stream(side)
            x[0].copy_(outs[-1])
            outs.append(binding.op_tree_attention(x[0][:B], *c, slot, cached, i32_one, mask[:B], 1, ks[layer], vs[layer]))
        binding.op_kv_commit(kc, vc, slot, cached, path, n_path, ks, vs)
        outs.append(binding.op_kv_load(kc[1], vc[1], rs, rp, ks[1], vs[1])[1])
        return outs

    def reset():
        for t in (kc, vc, ks, vs):
            t.zero_()

    i32_one = i32(np.arange(B + 1))
    want = None
    for _ in range(30):
        reset()
        got = chain(False)
        torch.cuda.synchronize()
        want = want or [g.clone() for g in got]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    m = mask.cpu().numpy()
    reset()
    binding.op_kv_store(src[1], src[2], kc[0], vc[0], rs, rp, ks[0], vs[0])
    ref, tol = attend64(src[0], kc[0], vc[0], ks[0], vs[0], slot.tolist(), cached.tolist(), first.tolist(), m, 1 / 8)
    check_attention(want[0], ref, tol)
    for fork in (False, True):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            held = chain(fork)
        for _ in range(5):
            reset()
            g.replay()
            torch.cuda.synchronize()
            attended = [h for i, h in enumerate(held) if not fork or i not in (0, 3)]
            assert all(torch.equal(a, b) for a, b in zip(attended, want))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: store, attention, load and commit
    in its last slot."""
    import torch
    S, K, P, D = 130, 4, 66000, 128
    assert S * K * P * D > 2 ** 32
    kc = torch.zeros((S, K, P, D), dtype=torch.int8, device="cuda")
    vc = torch.zeros((S, K, P, D), dtype=torch.int8, device="cuda")
    ks, vs = (torch.zeros((S, K, P), device="cuda") for _ in range(2))
    rng = np.random.default_rng(15)
    n = 6
    k = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).cuda()
    slot, pos = i32([S - 1] * n), i32(np.arange(P - n, P))
    binding.op_kv_store(k, v, kc, vc, slot, pos, ks, vs)
    k2, v2 = binding.op_kv_load(kc, vc, slot, pos, ks, vs)
    for a, b in ((k, k2), (v, v2)):
        step = a.abs().amax(-1, keepdim=True) / 127
        assert ((a - b).abs() <= step * 0.5001).all()
    mask = binding.tree_masks([-1, 0, 0, 2, 3, 4])
    q = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).cuda()
    got = binding.op_tree_attention(q, kc[S - 1:], vc[S - 1:], i32([0]), i32([P - n]), i32([0, n]),
                                    torch.from_numpy(mask).cuda(), n, ks[S - 1:], vs[S - 1:])
    same = binding.op_tree_attention(q, kc, vc, i32([S - 1]), i32([P - n]), i32([0, n]),
                                     torch.from_numpy(mask).cuda(), n, ks, vs)
    assert torch.equal(got, same) and got.abs().max() > 0
    before = [t[S - 1, :, P - 3].clone() for t in (kc, vc, ks, vs)]
    binding.op_kv_commit(kc, vc, i32([S - 1]), i32([P - n]), i32([[0, 3, -1, -1, -1, -1]]), i32([2]), ks, vs)
    for t, x in zip((kc, vc, ks, vs), before):
        assert torch.equal(t[S - 1, :, P - 5], x)


def test_binding_refuses():
    """Wrong devices, types, shapes and strides never reach the library."""
    import torch
    K, D, P = 2, 64, 40
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
    kc, vc = z(1, K, P, D), z(1, K, P, D)
    q, one, mask = z(3, K, D), i32([0]), z(3, t=torch.int64)
    first, idx = i32([0, 3]), i32([0, 0, 0])
    ok = dict(q=q, k_cache=kc, v_cache=vc, slot=one, cached=one, first=first, mask=mask, max_nodes=3)
    binding.op_tree_attention(**ok)
    for bad in (dict(q=q.cpu()), dict(q=q.double()), dict(q=q[:, :, ::2]), dict(k_cache=kc.transpose(1, 2)),
                dict(v_cache=vc[:, :1]), dict(v_cache=vc.half()), dict(slot=one.long()), dict(first=first[:1]),
                dict(mask=mask[:2]), dict(mask=mask.int()), dict(k_scale=z(1, K, P)), dict(out=z(3, K, D, t=torch.half)),
                dict(k_cache=kc.char(), v_cache=vc.char()), dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            binding.op_tree_attention(**{**ok, **bad})
    for bad in (dict(max_nodes=65), dict(max_nodes=0), dict(q=q.half()), dict(q=z(3, 3, D)),
                dict(scale=math.inf), dict(q=z(3, K, D + 4)[:, :, :D])):
        with pytest.raises((ValueError, binding.GPT2Error)):
            binding.op_tree_attention(**{**ok, **bad})
    for call in (lambda: binding.op_kv_store(q, q.half(), kc, vc, idx, idx), lambda: binding.op_kv_store(q, q, kc, vc, idx, one),
                 lambda: binding.op_kv_load(kc, vc, idx, idx, k=q), lambda: binding.op_kv_load(kc, vc, idx, idx, dtype=torch.int8),
                 lambda: binding.op_kv_commit(kc, vc, one, one, i32([0]), one),
                 lambda: binding.op_kv_commit(kc, vc, one, one, z(1, 65, t=torch.int32), one),
                 lambda: binding.op_verify_tree(z(3, 9), idx, idx, first, 3, 1.0),
                 lambda: binding.op_verify_tree(z(3, 9).half(), idx, idx, first, 3),
                 lambda: binding.op_verify_tree(z(3, 9), idx, idx, first, 3, workspace=z(4))):
        with pytest.raises((ValueError, binding.GPT2Error)):
            call()


# ---- verification -----------------------------------------------------------------------

def verify64(logits, tokens, parents, first, max_nodes, temperature, draft, ua, ud):
    """The walk in float64, sequence by sequence, as gpt2.h defines it.  Also
    returns how near any comparison came to its border (relative)."""
    V = logits.shape[1]
    near = math.inf
    res = []
    for b in range(len(first) - 1):
        f, n = first[b], min(first[b + 1] - first[b], max_nodes)
        if n == 0:
            res.append(([], -1))
            continue

        def dist(i):
            x = logits[f + i].astype(np.float64)
            if temperature == 0:
                return x if (x > -np.inf).any() else None
            if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
                return None
            e = np.exp((x - x.max()) / temperature)
            return e / e.sum()

        cur, path, p = 0, [0], dist(0)
        r = None if p is None else p.copy()
        while True:
            step = None
            for i in range(cur + 1, n):
                x = tokens[f + i]
                if parents[f + i] != cur or not 0 <= x < V or p is None:
                    continue
                if temperature == 0:
                    if int(np.nanargmax(p)) == x:
                        step = i
                        break
                    continue
                q = draft[f + cur].astype(np.float64) if draft is not None else np.eye(1, V, x)[0]
                lhs = float(ua[f + i]) * q[x]
                near = min(near, abs(lhs - r[x]) / max(lhs, r[x], 1e-300))
                if lhs < r[x]:
                    step = i
                    break
                r = np.maximum(r - q, 0)
                if r.sum() > 0:
                    r = r / r.sum()
            if step is None:
                break
            cur = step
            path.append(cur)
            p = dist(cur)
            r = None if p is None else p.copy()
        if p is None:
            res.append((path, -1))
        elif temperature == 0:
            res.append((path, int(np.nanargmax(p))))
        else:
            w = (r if r.sum() > 0 else p) / -np.log(ud[b].astype(np.float64))
            top = np.sort(w)[::-1]
            if V > 1:
                near = min(near, (top[0] - top[1]) / top[0])
            res.append((path, int(np.argmax(w))))
    return res, near


def uniform(rng, *shape):
    return ((rng.integers(0, 1 << 23, shape) + 0.5) * 2.0 ** -23).astype(np.float32)


def verify_inputs(rng, counts, V, width, spread=2.0):
    n = sum(counts)
    logits = (spread * rng.standard_normal((n, V))).astype(np.float32)
    dl = logits + rng.standard_normal((n, V))
    draft = np.exp(dl - dl.max(1, keepdims=True))
    draft = (draft / draft.sum(1, keepdims=True)).astype(np.float32)
    parents = [q for c in counts if c for q in random_tree(rng, c, width)]
    first = np.concatenate([[0], np.cumsum(counts)])
    tokens = np.zeros(n, np.int64)
    for b in range(len(counts)):
        for i in range(first[b], first[b + 1]):
            up = first[b] + max(parents[i], 0)
            tokens[i] = np.argmax(np.log(draft[up] + 1e-30) - np.log(-np.log(uniform(rng, V))))
    return logits, draft, tokens, np.array(parents), first


def run_verify(logits, tokens, parents, first, max_nodes, temperature, draft, ua, ud):
    import torch
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda() if x is not None else None
    path, n_path, nxt = binding.op_verify_tree(up(logits), i32(tokens), i32(parents), i32(first), max_nodes, temperature,
                                               up(draft), up(ua), up(ud))
    path, n_path, nxt = path.cpu().numpy(), n_path.cpu().numpy(), nxt.cpu().numpy()
    out = []
    for b in range(len(first) - 1):
        assert (path[b, n_path[b]:] == -1).all()
        out.append((path[b, :n_path[b]].tolist(), int(nxt[b])))
    return out


@pytest.mark.parametrize("temperature", [0.0, 0.7, 1.0])
@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("counts,V,width", [([6, 1, 0, 4, 6], 1003, 1), ([8, 8, 5], 50257, 3), ([64, 30], 517, 5),
                                            ([3, 2], 1, 1), ([5, 9], 8193, 2), ([16] * 40, 300, 4)])
def test_verify_walks_as_defined(counts, V, width, dense, temperature):
    """Chains and trees, with and without the draft's distributions, vocabularies
    of one, odd and large; no sequence without its decision clear of a border
    by 1e-5 (the fp32 sums are good to about 1e-6)."""
    rng = np.random.default_rng(V + width)
    logits, draft, tokens, parents, first = verify_inputs(rng, counts, V, width)
    n = len(tokens)
    for again in range(20):
        ua, ud = uniform(rng, n), uniform(rng, len(counts), V)
        want, near = verify64(logits, tokens, parents, first, max(counts), temperature, draft if dense else None, ua, ud)
        if near > 1e-5:
            break
    else:
        raise AssertionError("no draw of the random numbers is clear of the borders")
    got = run_verify(logits, tokens, parents, first, max(counts), temperature, draft if dense else None, ua, ud)
    assert got == want


def test_verify_edges():
    """-infinity, NaN and +infinity logits, tokens outside the vocabulary, a
    sibling's token twice, parents that do not come first, max_nodes below a
    sequence's nodes."""
    rng = np.random.default_rng(3)
    V = 700
    logits, draft, tokens, parents, first = verify_inputs(rng, [7] * 8, V, 2)
    parents[:7] = [-1, 0, 0, 0, 0, 0, 0]
    tokens[1:7] = tokens[1]                      # the same drafted token six times
    logits[7] = -np.inf                          # no choice at the root of sequence 1
    logits[14, 5] = np.nan
    logits[21, 9] = np.inf
    logits[28, 100:] = -np.inf                   # masked ids
    tokens[36:42] = [-1, V, V + 7, 1 << 30, 3, 4]
    parents[42:49] = [5, 0, 3, 2, -4, 4, 99]
    for temperature in (0.0, 0.9):
        for dense in (True, False):
            for mx in (7, 5, 1):
                ua, ud = uniform(rng, 56), uniform(rng, 8, V)
                d = draft if dense else None
                want, near = verify64(logits, tokens, parents, first, mx, temperature, d, ua, ud)
                assert near > 1e-5
                assert run_verify(logits, tokens, parents, first, mx, temperature, d, ua, ud) == want


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("low", [-np.inf, -3.3e38])
def test_verify_masked_children_among_siblings(low, dense):
    """Drafted tokens of probability zero (a logit of -infinity, or so far below
    the largest that the difference passes fp32's range) are rejected without
    touching what is left for their siblings."""
    rng = np.random.default_rng(30)
    V, B = 300, 24
    logits, draft, tokens, parents, first = verify_inputs(rng, [6] * B, V, 5)
    logits[:, ::2] = low
    logits[:, 1] += 3
    logits[:, 3] = logits[:, 1] - 0.25
    if low > -np.inf:
        logits[:, 1:4:2] += np.float32(3.3e38)
    parents = np.tile([-1, 0, 0, 0, 0, 0], B)
    tokens = np.tile([0, 1, 8, 3, 10, 3], B)
    for again in range(20):
        ua, ud = uniform(rng, 6 * B), uniform(rng, B, V)
        ua[1::6] = 1 - 2.0 ** -24
        d = draft if dense else None
        want, near = verify64(logits, tokens, parents, first, 6, 1.0, d, ua, ud)
        if near > 1e-5:
            break
    else:
        raise AssertionError("no draw of the random numbers is clear of the borders")
    assert run_verify(logits, tokens, parents, first, 6, 1.0, d, ua, ud) == want


@pytest.mark.parametrize("temperature", [3e38, 1.3e37, 2.0 ** 121, 5e-38])
def test_verify_extreme_temperatures(temperature):
    """With masked ids: the distribution over the others is flat, or on the
    highest."""
    rng = np.random.default_rng(31)
    logits, draft, tokens, parents, first = verify_inputs(rng, [5] * 6, 64, 2)
    logits[:, 5::7] = -np.inf
    if temperature < 1:                          # (the highest clear of the others)
        logits = np.round(logits * 4)
        logits[:, 3] = 90
    ua, ud = uniform(rng, 30), uniform(rng, 6, 64)
    want, near = verify64(logits, tokens, parents, first, 5, temperature, draft, ua, ud)
    assert near > 1e-5
    assert run_verify(logits, tokens, parents, first, 5, temperature, draft, ua, ud) == want


def test_verify_ties_take_the_lowest_id():
    V = 20000
    logits = np.zeros((2, V), np.float32)
    logits[0, [77, 9000, 19999]] = 2
    logits[1, [0, 8192]] = 2
    got = run_verify(logits, [0, 77], [-1, 0], [0, 2], 2, 0.0, None, None, None)
    assert got == [([0, 1], 0)]
    ud = np.full((1, V), 0.5, np.float32)        # equal noise: the race is decided by r, ties by id
    got = run_verify(logits, [0, 5], [-1, 0], [0, 2], 2, 1.0, None, np.array([0.5, 0.999999], np.float32), ud)
    assert got == [([0], 77)]


@pytest.mark.parametrize("V", [1, 7, 130, 8192, 20000, 50257])
def test_verify_greedy_takes_the_lowest_of_equals(V):
    """Equal highest logits anywhere in the row, zeros of both signs among them,
    next to NaN and -infinity."""
    rng = np.random.default_rng(V)
    n = 40
    logits = -rng.random((n, V)).astype(np.float32) - 1
    for i in range(n):
        at = rng.integers(0, V, 4)
        logits[i, at[3]] = (np.nan, -np.inf)[i % 2]
        if i % 3:
            logits[i, at[:3]] = 0.0
            logits[i, at[:3].min()] = -0.0
        else:
            logits[i, at[:3]] = 5.0
    got = run_verify(logits, np.zeros(n, int), -np.ones(n, int), np.arange(n + 1), 1, 0.0, None, None, None)
    for i in range(n):
        x = logits[i]
        ok = (x > -np.inf).any()
        assert got[i] == ([0], int(np.nanargmax(x)) if ok else -1)


def test_verify_gives_the_targets_distribution():
    """The first token a sequence gains (an accepted child's, or the drawn one)
    is distributed as softmax(logits / T) whatever the draft: chi-square of
    40,000 sequences with two drafted siblings each, V = 12 (11 degrees of
    freedom: 99.9% below 31.3)."""
    rng = np.random.default_rng(21)
    B, V, T = 40000, 12, 0.8
    row = (1.5 * rng.standard_normal(V)).astype(np.float32)
    dr = rng.random(V).astype(np.float32)
    dr /= dr.sum()
    logits = np.repeat(row[None], 3 * B, 0)
    draft = np.repeat(dr[None], 3 * B, 0).astype(np.float32)
    tokens = rng.choice(V, 3 * B, p=dr.astype(np.float64) / dr.sum(dtype=np.float64))
    parents = np.tile([-1, 0, 0], B)
    first = np.arange(B + 1) * 3
    p = np.exp(row.astype(np.float64) / T)
    p /= p.sum()
    for d in (draft, None):
        got = run_verify(logits, tokens, parents, first, 3, T, d, uniform(rng, 3 * B), uniform(rng, B, V))
        gained = [tokens[3 * b + path[1]] if len(path) > 1 else nxt for b, (path, nxt) in enumerate(got)]
        count = np.bincount(gained, minlength=V)
        chi2 = ((count - B * p) ** 2 / (B * p)).sum()
        assert chi2 < 31.3, (chi2, count / B, p)


def test_verify_streams_and_graphs():
    """The same workspace in two captured graphs replayed one after the other,
    and a call on another stream."""
    import torch
    rng = np.random.default_rng(22)
    V, counts = 5000, [4, 3]
    runs = []
    ws = torch.empty(binding.op_verify_tree_workspace(7, V), dtype=torch.uint8, device="cuda")
    for k in range(2):
        logits, draft, tokens, parents, first = verify_inputs(rng, counts, V, 2)
        ua, ud = uniform(rng, 7), uniform(rng, 2, V)
        want, near = verify64(logits, tokens, parents, first, 4, 1.0, draft, ua, ud)
        assert near > 1e-5
        args = [torch.from_numpy(logits).cuda(), i32(tokens), i32(parents), i32(first), 4, 1.0,
                torch.from_numpy(draft).cuda(), torch.from_numpy(ua).cuda(), torch.from_numpy(ud).cuda()]
        g = torch.cuda.CUDAGraph()
        binding.op_verify_tree(*args, workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = binding.op_verify_tree(*args, workspace=ws)
        runs.append((g, out, want, args))
    for k in (0, 1, 0):
        for t in runs[k][1]:
            t.fill_(123)
        runs[k][0].replay()
    torch.cuda.synchronize()
    for g, out, want, args in runs:
        path, n_path, nxt = (t.cpu().numpy() for t in out)
        assert [(path[b, :n_path[b]].tolist(), int(nxt[b])) for b in range(2)] == want
    s = torch.cuda.Stream()
    out = binding.op_verify_tree(*runs[0][3], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, runs[0][1]))


# ---- commit -----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("D", DIMS)
def test_commit_moves_the_accepted_rows(kind, D):
    """Paths of every kind in one call, three layers; entries that break a path
    end it; all other rows keep their bits."""
    import torch
    rng = np.random.default_rng(D)
    L, S, H, P, T = 3, 9, 2, 83, 64
    paths = [[0], [0, 1, 2, 3], [0, 2, 3, 7], list(range(0, 64, 2)), [0, 5, 4, 6], [0, 3, 70], [], [0, 63], [1, 2]]
    cached = [0, 5, 10, 19, 3, 0, 4, 30, 7]
    keep = [1, 4, 4, 32, 2, 2, 0, 1, 0]              # entries that count (the tail of a bad path does not)
    slot = rng.permutation(S)
    x = [make_cache(rng, kind, L * S, H, P, D) for _ in range(2)]
    caches = [t for c, s in x for t in (c, s) if t is not None]
    shaped = [t.view(L, S, H, *t.shape[2:]) for t in caches]
    kc, vc = shaped[0], shaped[len(shaped) // 2]
    ks, vs = (shaped[1], shaped[3]) if len(shaped) == 4 else (None, None)
    want = [raw(t).reshape(L, S, H, P, -1).copy() for t in shaped]
    orig = [w.copy() for w in want]
    p = np.full((S, T), -1)
    for b, path in enumerate(paths):
        p[b, :len(path)] = path
        for w, o in zip(want, orig):
            for i in range(keep[b]):
                w[:, slot[b], :, cached[b] + i] = o[:, slot[b], :, cached[b] + path[i]]
    binding.op_kv_commit(kc, vc, i32(slot), i32(cached), i32(p), i32([len(q) for q in paths]), ks, vs)
    for t, w in zip(shaped, want):
        assert np.array_equal(raw(t).reshape(w.shape), w)
    # slots and lengths outside the cache are skipped
    binding.op_kv_commit(kc, vc, i32([-1, S, 1, 2]), i32([0, 0, -3, P]), i32([[0, 2]] * 4), i32([2] * 4), ks, vs)
    for t, w in zip(shaped, want):
        assert np.array_equal(raw(t).reshape(w.shape), w)
