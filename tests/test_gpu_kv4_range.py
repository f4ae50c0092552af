"""The attention's range: value scales far apart, logits far below zero, large logits close together."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import dev, sequences
from tests.test_gpu_kv4_attention import attend, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def peak_of(geo, cache, table_row, n, q, scale, first):
    """Largest weight times value scale, over the keys a row sees and their groups, [T, H]: rows at positions first + t."""
    T, H, _ = q.shape
    per = geo.q_heads // geo.kv_heads
    out = np.zeros((T, H))
    for h in range(geo.kv_heads):
        K, _ = o.gather(geo, cache, table_row, h, n)
        s = np.zeros(n)
        for j in range(n):
            at = geo.base(int(table_row[j // geo.page]), h, j % geo.page) + 32 * geo.D + 128 * geo.G + 4 * geo.G * (j % 32)
            s[j] = (cache[at:at + 4 * geo.G].copy().view("<u4") & 0xFFFF).astype(np.uint16).view(np.float16).max()
        for g in range(h * per, (h + 1) * per):
            for t in range(T):
                m = first + t + 1
                x = scale * (K[:m] @ q[t, g].astype(np.float64))
                p = np.exp(x - x.max())
                out[t, g] = (p * s[:m]).max() / p.sum()
    return out


def tolerance(size, reach, keys, D, f16, peak):
    """As the oracle's bound, but what a product p s' loses below fp16's normal range (2^-25 a key, codes up to 15) set
    beside the row's own largest product: the running reference keeps that at 2^9 or above.  fp32 calls: p s' in
    two fp16 parts, 2^-22 relative."""
    tol = o.attention_tolerance(size, reach, keys, D, f16, 0.0) + keys * 15 * 2.0 ** -34 * peak[..., None]
    return tol + (0 if f16 else size * 2.0 ** -22)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("new", [1, 6, 20, 40])
@pytest.mark.parametrize("others", [-4, 8])
def test_keys_with_nearly_all_the_weight_and_small_values(mnb, others, new, group, dt):
    """In blocks that every row sees whole, beside keys of far larger value scales: exact to their own size."""
    rng = np.random.default_rng((970, new, group, others + 50))
    past, D, H = 96, 128, 2
    n = past + new
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(H, 1, D, group, 32, pages)
    cache, _ = make_cache(rng, geo, table, [n], k_scale=0.05)
    NG, u = D // group, rng.choice([-1.0, 1.0], D)
    for j in range(n):                                # the others' value scales
        at = geo.base(int(table[0, j // 32]), 0, j % 32) + 32 * D + 128 * NG + 4 * NG * (j % 32)
        cache[at:at + 4 * NG] = np.full(NG, int(np.float16(2.0 ** others).view(np.uint16)) | (8 << 16), "<u4").view(np.uint8)
    for star, ks in ((40, 1.0), (41, 0.995), (73, 0.99)):     # alike, so that no weight is a power of two of another
        small = (2.0 ** -20 * rng.uniform(1, 2, NG)).astype(np.float16)
        o.store(geo, cache, int(table[0, star // 32]), 0, star % 32, False, (8 + 7 * u).astype(int), np.full(NG, ks, np.float16),
                np.full(NG, 8))
        o.store(geo, cache, int(table[0, star // 32]), 0, star % 32, True, rng.integers(0, 16, D), small, np.full(NG, 7))
    q = (0.5 * rng.normal(size=(new, H, D)) + u).astype(np.float16 if dt == "f16" else np.float32)
    w, _, size, reach = o.attention(geo, cache, table, [n], [0, new], q, D ** -0.5)
    assert np.abs(w).max() < 2.0 ** -15               # the small keys' values
    tol = tolerance(size, reach, n, D, dt == "f16", peak_of(geo, cache, table[0], n, q, D ** -0.5, past))
    err = np.abs(G.host(attend(mnb, geo, cache, table, [n], [0, new], q, D ** -0.5)[0]) - w)
    assert (err <= tol).all(), "worst %.3g of the bound" % float((err / tol).max())


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("rise", [0, 1])
@pytest.mark.parametrize("new", [1, 7, 30, 60])
def test_value_scales_of_every_size(mnb, new, rise, dt):
    """Value scales over fp16's whole range, with level logits or ones that rise along the keys, bounded by each row's own
    largest product."""
    rng = np.random.default_rng((971, new, rise))
    n, D = 260, 128
    table, pages = sequences(rng, [n], 64)
    geo = o.Geometry(2, 1, D, 64, 64, pages)
    cache, _ = make_cache(rng, geo, table, [n], k_scale=0.2)
    meta = cache.reshape(-1, geo.B)[:, 32 * D:].copy().view("<u4")
    for j in range(n):
        row, at = int(table[0, j // 64]) * 2 + j % 64 // 32, j % 32 * 2
        s = np.float16(2.0) ** rng.integers(-24, 9, 2).astype(np.float16)
        ks = np.float16(0.05 + rise * 0.8 * j / n)
        for g in range(2):
            meta[row, at + g] = (int(meta[row, at + g]) & 0xFFFF0000) | int(ks.view(np.uint16))
            meta[row, 64 + at + g] = (int(meta[row, 64 + at + g]) & 0xFFFF0000) | int(s[g].view(np.uint16))
    cache.reshape(-1, geo.B)[:, 32 * D:] = meta.view(np.uint8)
    q = (1.5 * rng.normal(size=(new, 2, D))).astype(np.float16 if dt == "f16" else np.float32)
    w, _, size, reach = o.attention(geo, cache, table, [n], [0, new], q, D ** -0.5)
    tol = tolerance(size, reach, n, D, dt == "f16", peak_of(geo, cache, table[0], n, q, D ** -0.5, n - new))
    err = np.abs(G.host(attend(mnb, geo, cache, table, [n], [0, new], q, D ** -0.5)[0]) - w)
    assert (err <= tol).all(), "worst %.3g of the bound" % float((err / tol).max())


@pytest.mark.parametrize("new", [1, 8, 16, 40])
@pytest.mark.parametrize("split", [False, True])
def test_logits_far_below_zero(mnb, new, split):
    """fp32 queries whose logits are all one large negative number: equal weights, not a row that sees nothing."""
    rng = np.random.default_rng(972)
    n, D = 300, 128
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(1, 1, D, 128, 32, pages)
    cache, _ = make_cache(rng, geo, table, [n])
    for j in range(n):
        o.store(geo, cache, int(table[0, j // 32]), 0, j % 32, False, np.full(D, 15), np.ones(1, np.float16), np.zeros(1, int))
    V = o.gather(geo, cache, table[0], 0, n)[1]
    q = np.full((new, 1, D), -1e31, np.float32)
    got, lse = attend(mnb, geo, cache, table, [n], [0, new], q, 0.125, max_kv=3000 if split else n)
    got, lse = G.host(got), G.host(lse)
    x = -0.125 * 15 * D * float(np.float32(1e31))
    for t in range(new):
        seen = V[:n - new + t + 1]
        # equal logits, so equal weights; the sums in fp32, the weights times the scales in two fp16 parts
        tol = np.abs(seen).mean(0) * ((n + 64) * o.EPS32 + 2.0 ** -22) + 2.0 ** -30
        assert (np.abs(got[t, 0] - seen.mean(0)) <= tol).all(), t
        assert abs(lse[t, 0] - x) <= abs(x) * (D + 16) * o.EPS32, t


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("new", [1, 3, 8, 16, 40, 150])
def test_a_row_s_bits_come_from_its_own_keys(mnb, new, split, dt):
    """Neither what lies in places without a token, nor keys that a row does not see, nor the rows beside it decide a
    bit of it."""
    t = G.torch()
    rng = np.random.default_rng((974, new))
    past, D, H = 100, 128, 2
    n = past + new
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(H, 1, D, 64, 32, pages)
    cache, _ = make_cache(rng, geo, table, [n], k_scale=0.5)     # logits over a wide range: references move often
    q = (2.0 * rng.normal(size=(new, H, D))).astype(np.float16 if dt == "f16" else np.float32)
    kw = dict(max_kv=3000 if split else n)
    want, _ = attend(mnb, geo, cache, table, [n], [0, new], q, D ** -0.5, **kw)
    words = np.array([0x00080000, 0x00087BFF, 0x00087C00, 0x00087E00, 0xFFFFFFFF], np.uint32)
    for word in words:                                # places after the last token, keys and values
        other = cache.copy()
        for j in range(n, -(-n // 32) * 32):
            at = geo.base(int(table[0, j // 32]), 0, j % 32) + 32 * D + 8 * (j % 32)
            other[at:at + 8] = other[at + 256:at + 264] = np.array([word, word], "<u4").view(np.uint8)
        got, _ = attend(mnb, geo, other, table, [n], [0, new], q, D ** -0.5, **kw)
        assert t.equal(got, want), hex(word)
    if new == 1:
        return
    for word in words:                                # the last key, which only the last token sees
        other = cache.copy()
        at = geo.base(int(table[0, (n - 1) // 32]), 0, (n - 1) % 32) + 32 * D + 8 * ((n - 1) % 32)
        other[at:at + 8] = other[at + 256:at + 264] = np.array([word, word], "<u4").view(np.uint8)
        got, _ = attend(mnb, geo, other, table, [n], [0, new], q, D ** -0.5, **kw)
        assert t.equal(got[:-1], want[:-1]), hex(word)
    for value in (np.inf, np.nan, 3e4, 0.0):          # one row of queries
        other = q.copy()
        other[new // 2, 1] = value
        got, _ = attend(mnb, geo, cache, table, [n], [0, new], other, D ** -0.5, **kw)
        keep = t.ones((new, H), dtype=t.bool, device="cuda")
        keep[new // 2, 1] = False
        assert t.equal(got[keep], want[keep]), value


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("size", [2 ** 20, 2 ** 22, 2 ** 24, 2 ** 26])
@pytest.mark.parametrize("new", [1, 6, 16, 30, 40])
def test_large_logits_that_differ_little(mnb, new, size, dt):
    """Logits of `size` (in units of log2) apart by a few units, beside value scales just below a power of two: whatever is
    left of the differences, the outputs are means of the values."""
    rng = np.random.default_rng((975, new, size))
    D, n, half = 128, 500, 64
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(1, 1, D, D, 32, pages)
    cache, _ = make_cache(rng, geo, table, [n])
    u = rng.choice([-1, 1], half)
    V = np.zeros((n, D))
    for j in range(n):
        codes = np.concatenate([8 + 4 * u, rng.integers(0, 16, half)])
        o.store(geo, cache, int(table[0, j // 32]), 0, j % 32, False, codes, np.full(1, 8, np.float16), np.full(1, 8))
        s = np.float16(0.9995 * 2.0 ** rng.integers(-3, 4))
        vc = rng.integers(0, 16, D)
        o.store(geo, cache, int(table[0, j // 32]), 0, j % 32, True, vc, np.full(1, s, np.float16), np.full(1, 8))
        V[j] = (vc - 8.0) * float(s)
    scale = size * np.log(2.0) / (half * 4 * 8 * 6e4)
    q = np.zeros((new, 1, D), np.float16 if dt == "f16" else np.float32)
    q[:, 0, :half] = 6e4 * u
    # codes less 8 have a deviation of 4.6: logits apart by about 6
    q[:, 0, half:] = rng.normal(size=(new, half)) * 6 / (scale * 1.44 * 8 * 4.6 * 8)
    out, lse = attend(mnb, geo, cache, table, [n], [0, new], q, scale)
    got, lse = G.host(out)[:, 0], G.host(lse)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    lo, hi = np.minimum.accumulate(V, 0)[n - new:], np.maximum.accumulate(V, 0)[n - new:]
    slack = 2.0 ** -9 * np.maximum(np.abs(lo), np.abs(hi))     # p s' and the output rounded to fp16, sums in fp32
    assert (got >= lo - slack).all() and (got <= hi + slack).all()
    assert (np.abs(lse / np.log(2.0) - size) <= 64 + size * 2.0 ** -15).all()
