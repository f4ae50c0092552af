"""The paged 4-bit cache on the GPU: what append writes, byte for byte against
the oracle's binary32 steps, and what read gives back."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def dev(a):
    return G.torch().from_numpy(np.ascontiguousarray(a)).cuda()


def sequences(rng, lens, page, spare=2):
    """A page table with the pages in random order, garbage past each sequence, and the number of pages."""
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = rng.integers(-5, 1 << 30, (len(lens), max(need + [1]) + 1)).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def desc_of(mnb, geo):
    return mnb.kv4_desc(geo.q_heads, geo.kv_heads, geo.D, geo.group, geo.page, geo.num_pages)


CASES = [  # D, group, page, q heads, kv heads, new tokens, past
    (64, 64, 32, 4, 2, [1, 1, 1], [0, 31, 32]),
    (64, 32, 64, 3, 3, [5, 0, 40], [10, 7, 63]),
    (128, 128, 64, 8, 2, [1], [100]),
    (128, 128, 32, 8, 1, [33, 1, 2, 64], [0, 5, 30, 31]),
    (128, 64, 256, 4, 4, [300], [0]),
    (128, 32, 128, 6, 2, [17, 3], [250, 0]),
    (256, 128, 64, 2, 1, [9, 70], [1, 60]),
    (256, 64, 32, 5, 5, [3], [29]),
    (256, 32, 64, 2, 2, [2, 1], [62, 0]),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("rot", ["none", "all", "half", "interleaved"])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:5])) for c in CASES])
def test_append_writes_the_documented_bytes(mnb, case, rot, dt):
    t = G.torch()
    D, group, page, H, Hkv, new, past = case
    rng = np.random.default_rng((920, D, group, page, H))
    lens = [n + p for n, p in zip(new, past)]
    table, pages = sequences(rng, lens, page)
    geo = o.Geometry(H, Hkv, D, group, page, pages)
    T = sum(new)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    kind = np.float16 if dt == "f16" else np.float32
    # one projection's output: q, k and v are slices of its rows, at an odd element
    qkv = rng.normal(size=(T, (H + 2 * Hkv) * D + 3)).astype(kind)
    qkv *= np.exp(rng.normal(size=(T, 1))).astype(kind)
    parts = [qkv[:, 3:3 + H * D], qkv[:, 3 + H * D:3 + (H + Hkv) * D], qkv[:, 3 + (H + Hkv) * D:]]
    q, k, v = [p.reshape(T, -1, D) for p in parts]
    R = 0 if rot == "none" else D // 2 if rot == "half" else D
    cos = sin = None
    if R:
        ang = rng.uniform(0, 6.3, (max(lens) - 2 if max(lens) > 4 else 4, R // 2))    # the last positions share a row
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    want = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    cache = dev(want)
    pos = o.append(geo, want, table, lens, q_start, k, v, cos, sin, R, rot == "interleaved")
    dq = dev(qkv)
    views = [dq[:, 3:3 + H * D].unflatten(1, (H, D)), dq[:, 3 + H * D:3 + (H + Hkv) * D].unflatten(1, (Hkv, D)),
             dq[:, 3 + (H + Hkv) * D:].unflatten(1, (Hkv, D))]
    q_out = t.empty((T, H, D), dtype=dq.dtype, device="cuda")
    kl = np.array(lens, np.int32)
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, views[1], views[2], dev(table), dev(kl), dev(q_start),
                       cos=None if not R else dev(cos), sin=None if not R else dev(sin), rotary_dim=R,
                       interleaved=rot == "interleaved", q=views[0], q_out=q_out)
    got = cache.cpu().numpy()
    assert (got == want).all(), "%d of %d bytes differ" % ((got != want).sum(), want.size)
    wq = o.rotate(q, pos, cos, sin, R, rot == "interleaved").astype(kind)
    assert (q_out.cpu().numpy() == wq).all()

    # read the same rows back
    ko, vo = (t.full((T, Hkv, D), 9.0, dtype=dq.dtype, device="cuda") for _ in range(2))
    mnb.mnb_kv4_read(desc_of(mnb, geo), cache, dev(table), dev(kl), dev(q_start), ko, vo)
    for b in range(len(lens)):
        for h in range(Hkv):
            K, V = o.gather(geo, want, table[b], h, lens[b])
            rows = slice(q_start[b], q_start[b + 1])
            assert (ko[rows, h].cpu().numpy() == K[past[b]:].astype(kind)).all()
            assert (vo[rows, h].cpu().numpy() == V[past[b]:].astype(kind)).all()


def test_one_token_each_without_q_start(mnb):
    rng = np.random.default_rng(921)
    lens = [1, 33, 64, 100, 7]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(2, 2, 64, 32, 32, pages)
    k, v = (rng.normal(size=(5, 2, 64)).astype(np.float32) for _ in range(2))
    want = np.zeros(geo.bytes, np.uint8)
    o.append(geo, want, table, lens, list(range(6)), k, v)
    cache = dev(np.zeros(geo.bytes, np.uint8))
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), dev(table), dev(np.array(lens, np.int32)))
    assert (cache.cpu().numpy() == want).all()


def test_places_that_do_not_exist_are_not_written(mnb):
    """Negative positions, pages outside the cache, tokens past the table, rows past the last sequence."""
    t = G.torch()
    rng = np.random.default_rng(922)
    page = 32
    table = np.array([[1, -1], [0, 99], [3, 2]], np.int32)
    geo = o.Geometry(1, 1, 128, 128, page, 4)
    lens, new = [40, 33, 80], [12, 2, 20]
    lens[1] = 1                                        # two new tokens, one of them at position -1
    q_start = np.array([0, 12, 14, 34], np.int32)
    T = 36                                             # two rows past the last sequence
    k, v = (rng.normal(size=(T, 1, 128)).astype(np.float16) for _ in range(2))
    want = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    cache = dev(want)
    o.append(geo, want, table, lens, q_start, k, v)
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), dev(table), dev(np.array(lens, np.int32)), dev(q_start))
    assert (cache.cpu().numpy() == want).all()
    ko = t.full((T, 1, 128), 5.0, dtype=t.float16, device="cuda")
    mnb.mnb_kv4_read(desc_of(mnb, geo), cache, dev(table), dev(np.array(lens, np.int32)), dev(q_start), k_out=ko)
    got = G.host(ko)
    pos = o.positions(lens, q_start, T)
    for r in range(T):
        b = int(np.searchsorted(q_start[1:], r, side="right"))
        there = b < 3 and 0 <= pos[r] < 64 and 0 <= table[b, pos[r] // page] < 4
        if not there:
            assert (got[r] == 0).all(), r


def test_bad_values_stay_in_their_group(mnb):
    t = G.torch()
    rng = np.random.default_rng(923)
    table, pages = sequences(rng, [3], 32)
    geo = o.Geometry(1, 1, 128, 32, 32, pages)
    k, v = (rng.normal(size=(3, 1, 128)).astype(np.float32) for _ in range(2))
    k[0, 0, 40], k[1, 0, 100], v[2, 0, 3], v[1, 0, 64] = np.nan, np.inf, -np.inf, 3e6
    k[2] = 0
    v[0, 0, :32] = 1e-9                                # below the smallest scale
    cache = dev(np.zeros(geo.bytes, np.uint8))
    args = (desc_of(mnb, geo), cache)
    seq = (dev(table), dev(np.array([3], np.int32)), dev(np.array([0, 3], np.int32)))
    mnb.mnb_kv4_append(*args, dev(k), dev(v), *seq)
    ko, vo = (t.empty((3, 1, 128), device="cuda") for _ in range(2))
    mnb.mnb_kv4_read(*args, *seq, ko, vo)
    K, V = G.host(ko)[:, 0].reshape(3, 4, 32), G.host(vo)[:, 0].reshape(3, 4, 32)
    nan = np.zeros((2, 3, 4), bool)
    nan[0, 0, 1] = nan[0, 1, 3] = nan[1, 2, 0] = nan[1, 1, 2] = True
    assert (np.isnan(K).all(-1) == nan[0]).all() and (np.isnan(K).any(-1) == nan[0]).all()
    assert (np.isnan(V).all(-1) == nan[1]).all() and (np.isnan(V).any(-1) == nan[1]).all()
    assert (K[2] == 0).all() and (V[0, 0] == 0).all()


def test_many_sequences_are_found(mnb):
    """More sequences than the search's lanes, empty ones among them, one head."""
    rng = np.random.default_rng(924)
    new = rng.integers(0, 3, 700)
    lens = (new + rng.integers(0, 20, 700)).astype(np.int32)
    table, pages = sequences(rng, [int(n) for n in lens], 32)
    geo = o.Geometry(1, 1, 64, 64, 32, pages)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(q_start[-1])
    k, v = (rng.normal(size=(T, 1, 64)).astype(np.float16) for _ in range(2))
    want = np.zeros(geo.bytes, np.uint8)
    o.append(geo, want, table, lens, q_start, k, v)
    cache = dev(np.zeros(geo.bytes, np.uint8))
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), dev(table), dev(lens), dev(q_start))
    assert (cache.cpu().numpy() == want).all()


@pytest.mark.parametrize("new", [[511], [512], [513], [700, 1, 600]])
def test_prompts_longer_than_a_round_of_workgroups(mnb, new):
    """Every token is taken once where runs of them go to one XCD, and those past the last whole round."""
    t = G.torch()
    rng = np.random.default_rng((926, sum(new)))
    lens = np.array([n + 5 for n in new], np.int32)
    table, pages = sequences(rng, [int(n) for n in lens], 32)
    geo = o.Geometry(2, 1, 64, 64, 32, pages)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(q_start[-1])
    q, k, v = (rng.normal(size=(T, h, 64)).astype(np.float16) for h in (2, 1, 1))
    want = np.zeros(geo.bytes, np.uint8)
    o.append(geo, want, table, lens, q_start, k, v)
    cache = dev(np.zeros(geo.bytes, np.uint8))
    q_out = t.full((T, 2, 64), 9.0, dtype=t.float16, device="cuda")
    seq = (dev(table), dev(lens), dev(q_start))
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), *seq, q=dev(q), q_out=q_out)
    assert (cache.cpu().numpy() == want).all() and (q_out.cpu().numpy() == q).all()
    ko, vo = (t.full((T, 1, 64), 9.0, dtype=t.float16, device="cuda") for _ in range(2))
    mnb.mnb_kv4_read(desc_of(mnb, geo), cache, *seq, ko, vo)
    for b in range(len(new)):
        K, V = o.gather(geo, want, table[b], 0, int(lens[b]))
        rows = slice(q_start[b], q_start[b + 1])
        assert (ko[rows, 0].cpu().numpy() == K[5:].astype(np.float16)).all()
        assert (vo[rows, 0].cpu().numpy() == V[5:].astype(np.float16)).all()


def test_pages_past_four_gigabytes(mnb):
    """A page whose offset passes 32 bits."""
    t = G.torch()
    pages = 4 * 1024 * 1024 * 1024 // (2 * 32 * 128 + 512) + 700
    geo = o.Geometry(2, 2, 128, 128, 32, pages)
    d = desc_of(mnb, geo)
    assert mnb.mnb_kv4_cache_bytes(d) == geo.bytes > 1 << 32
    cache = t.zeros(geo.bytes, dtype=t.uint8, device="cuda")
    rng = np.random.default_rng(925)
    k, v = (rng.normal(size=(2, 2, 128)).astype(np.float16) for _ in range(2))
    table = np.array([[pages - 1]], np.int32)
    seq = (dev(table), dev(np.array([2], np.int32)), dev(np.array([0, 2], np.int32)))
    mnb.mnb_kv4_append(d, cache, dev(k), dev(v), *seq)
    small = o.Geometry(2, 2, 128, 128, 32, 1)
    want = np.zeros(small.bytes, np.uint8)
    o.append(small, want, np.array([[0]]), [2], [0, 2], k, v)
    assert (cache[-small.bytes:].cpu().numpy() == want).all()
    assert int(cache[:-small.bytes].count_nonzero()) == 0
    ko, vo = (t.empty((2, 2, 128), dtype=t.float16, device="cuda") for _ in range(2))
    mnb.mnb_kv4_read(d, cache, *seq, ko, vo)
    assert (G.host(ko)[:, 1] == o.gather(small, want, [0], 1, 2)[0].astype(np.float16)).all()
    out = t.empty((2, 2, 128), dtype=t.float16, device="cuda")
    mnb.mnb_attention_kv4(d, cache, dev(k), *seq, 2, 2, out, 0.1)
    w, _, size, reach = o.attention(small, want, np.array([[0]]), [2], [0, 2], k, 0.1)
    assert (np.abs(G.host(out) - w) <= o.attention_tolerance(size, reach, 2, 128, True, 16.0)).all()
