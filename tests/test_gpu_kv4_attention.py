"""Attention over the paged 4-bit cache on the GPU against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import desc_of, dev, sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def make_cache(rng, geo, table, lens, v_scale=0.15, k_scale=0.3):
    """Random codes; scales and zero points of a real cache in every token's place, and garbage (NaN, infinite and
    huge scales, zero points with all bits set) in places that hold no token."""
    nb = geo.bytes // geo.B
    cache = rng.integers(0, 256, (nb, geo.B), dtype=np.uint8)
    s = np.exp(0.4 * rng.normal(size=(nb, 2, 32 * geo.G)))
    s[:, 0] *= k_scale
    s[:, 1] *= v_scale
    z = rng.integers(4, 12, (nb, 2, 32 * geo.G)).astype(np.uint32)
    good = s.astype(np.float16).view(np.uint16).astype(np.uint32) | (z << 16)
    bad = rng.choice(np.array([0xFFFFFFFF, 0x00007C00, 0xFFFFFC00, 0x00007BFF, 0x000F7E00], np.uint32), good.shape)
    live = np.zeros((geo.num_pages, geo.page), bool)
    for b, n in enumerate(lens):
        for p in range(n):
            live[table[b, p // geo.page], p % geo.page] = True
    # [page, head, block, token] -> per block rows
    keep = np.broadcast_to(live.reshape(geo.num_pages, 1, geo.page // 32, 32, 1),
                           (geo.num_pages, geo.kv_heads, geo.page // 32, 32, geo.G)).reshape(nb, 1, 32 * geo.G)
    meta = np.where(keep, good, bad).astype("<u4")
    cache[:, 32 * geo.D:] = meta.reshape(nb, -1).view(np.uint8)
    vmax = float(s[:, 1].max()) * 15
    return cache.reshape(-1), vmax


def attend(mnb, geo, cache, table, lens, q_start, q, scale, max_q=None, max_kv=None, causal=True, window=0, want_lse=True,
           stream=None):
    t = G.torch()
    d = desc_of(mnb, geo)
    dq = dev(q) if isinstance(q, np.ndarray) else q
    T = dq.shape[0]
    new = np.diff(q_start)
    max_q = int(new.max()) if max_q is None else max_q
    max_kv = int(max(lens)) if max_kv is None else max_kv
    n = mnb.mnb_attention_kv4_workspace_bytes(d, len(lens), T, max_q, max_kv)
    ws = t.full((max(n, 256),), 0xFF, dtype=t.uint8, device="cuda")      # NaN to whatever reads it unwritten
    out = t.full(tuple(dq.shape), 7.0, dtype=dq.dtype, device="cuda")
    lse = t.full(tuple(dq.shape[:2]), 7.0, device="cuda") if want_lse else None
    mnb.mnb_attention_kv4(d, dev(cache) if isinstance(cache, np.ndarray) else cache, dq, dev(table),
                          dev(np.array(lens, np.int32)), dev(np.array(q_start, np.int32)), max_q, max_kv, out, scale,
                          causal=causal, window=window, lse=lse, workspace=ws, workspace_bytes=n, stream=stream)
    return out, lse


def check(mnb, geo, cache, vmax, table, lens, q_start, q, scale, causal=True, window=0, max_kv=None, **kw):
    out, lse = attend(mnb, geo, cache, table, lens, q_start, q, scale, causal=causal, window=window, max_kv=max_kv, **kw)
    w, wl, size, reach = o.attention(geo, cache, table, lens, q_start, q, scale, causal, window, max_kv)
    f16 = q.dtype == np.float16
    keys = max(max(lens), 1)
    tol = o.attention_tolerance(size, reach, keys, geo.D, f16, vmax)
    err = np.abs(G.host(out) - w)
    assert np.isfinite(G.host(out)).all()
    assert (err <= tol).all(), "worst %.3g of the bound" % float((err / tol).max())
    gl = G.host(lse)
    empty = np.isneginf(wl)
    assert (np.isneginf(gl) == empty).all() and (G.host(out)[empty] == 0).all()
    lt = o.lse_tolerance(np.where(empty, 0, wl), reach, keys, geo.D)
    assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, wl)) <= lt).all()
    return out


CASES = [  # D, group, page, q heads, kv heads, new tokens, cached with them
    (128, 128, 64, 4, 1, [1], [1]),
    (128, 128, 64, 8, 2, [1, 1, 1], [33, 64, 200]),
    (128, 64, 32, 6, 2, [1, 1], [1000, 1]),
    (128, 32, 128, 2, 2, [1, 3, 2], [130, 31, 97]),
    (64, 64, 32, 8, 1, [2, 2], [70, 300]),
    (64, 32, 256, 3, 3, [5], [260]),
    (256, 128, 64, 4, 2, [1, 2], [90, 33]),
    (256, 64, 32, 2, 1, [4], [65]),
    (256, 32, 32, 2, 1, [1], [40]),
    (128, 128, 64, 4, 1, [8, 5], [150, 9]),          # 32 and 20 rows
    (128, 64, 64, 8, 2, [20, 7], [84, 200]),         # rows over several tiles
    (128, 128, 32, 2, 2, [70, 1, 0, 33], [70, 64, 10, 133]),
    (64, 32, 64, 4, 2, [65], [129]),
    (256, 64, 64, 2, 1, [40], [100]),
    (256, 32, 64, 2, 1, [40], [100]),
    (128, 32, 32, 12, 1, [30], [50]),                # a group of 12 heads
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("mask", ["causal", "full", "window"])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:5] + (c[5][0], c[6][0]))) for c in CASES])
def test_against_the_oracle(mnb, case, mask, dt):
    D, group, page, H, Hkv, new, lens = case
    rng = np.random.default_rng((930, D, group, page, H, lens[0]))
    table, pages = sequences(rng, lens, page)
    geo = o.Geometry(H, Hkv, D, group, page, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (1.5 * rng.normal(size=(q_start[-1], H, D))).astype(np.float16 if dt == "f16" else np.float32)
    check(mnb, geo, cache, vmax, table, lens, q_start, q, D ** -0.5, causal=mask != "full",
          window=37 if mask == "window" else 0)


SPLIT = [  # D, group, q heads, kv heads, new tokens, cached with them
    (128, 128, 4, 2, [1, 1], [1500, 300]),           # few rows, up to 16 splits
    (64, 64, 2, 1, [3], [4900]),                     # few rows, more
    (256, 64, 4, 1, [1, 2, 0], [5100, 33, 0]),
    (128, 64, 3, 1, [40, 2], [1300, 700]),           # many rows, up to 16
    (64, 32, 2, 1, [35], [4500]),                    # many rows, more
    (256, 128, 2, 1, [20], [4400]),
    (128, 128, 8, 8, [520, 3], [1100, 1099]),        # so many that a split takes 512 keys
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("mask", ["causal", "full", "window"])
@pytest.mark.parametrize("case", SPLIT, ids=["-".join(map(str, c[:4] + (c[4][0], c[5][0]))) for c in SPLIT])
def test_keys_shared_between_workgroups(mnb, case, mask, dt):
    """Every form of the join: the splits of a row hold all, some or none of its keys."""
    D, group, H, Hkv, new, lens = case
    rng = np.random.default_rng((939, D, H, lens[0]))
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(H, Hkv, D, group, 64, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (1.5 * rng.normal(size=(q_start[-1], H, D))).astype(np.float16 if dt == "f16" else np.float32)
    check(mnb, geo, cache, vmax, table, lens, q_start, q, D ** -0.5, causal=mask != "full",
          window=600 if mask == "window" else 0)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_rows_that_see_nothing(mnb, dt):
    """Empty sequences, new tokens before position 0, and rows beside them that see keys."""
    rng = np.random.default_rng(931)
    lens, new = [0, 5, 40, 0], [2, 9, 3, 0]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(4, 2, 128, 128, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = rng.normal(size=(14, 4, 128)).astype(np.float16 if dt == "f16" else np.float32)
    check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1)
    check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, causal=False)
    # the same through many splits
    check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, max_kv=5000)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_a_wide_range_of_logits_and_scales(mnb, new, dt):
    """A first key with nearly all the weight and a near-zero value, logits that rise along the keys, value scales
    from the smallest to far above one, zero scales."""
    rng = np.random.default_rng(932)
    n, D = 400, 128
    table, pages = sequences(rng, [n], 64)
    geo = o.Geometry(2, 1, D, 64, 64, pages)
    cache, _ = make_cache(rng, geo, table, [n])
    blocks = cache.reshape(-1, geo.B)
    meta = blocks[:, 32 * D:].copy().view("<u4")
    vs = np.float16(2.0) ** rng.integers(-24, 9, (meta.shape[0], 64)).astype(np.float16)
    vs[rng.random(vs.shape) < 0.1] = 0
    meta[:, 64:] = (meta[:, 64:] & np.uint32(0xFFFF0000)) | vs.astype(np.float16).view(np.uint16)
    ks = np.linspace(0.02, 1.0, n).astype(np.float16)
    for p in range(n):
        row = int(table[0, p // 64]) * 2 + p % 64 // 32
        for g in range(2):
            at = p % 32 * 2 + g
            meta[row, at] = (int(meta[row, at]) & 0xFFFF0000) | int(ks[p].view(np.uint16))
            if p == 0:
                meta[row, 64 + at] = int(np.float16(2.0 ** -20).view(np.uint16)) | (8 << 16)
    blocks[:, 32 * D:] = meta.view(np.uint8)
    q = (2.0 * rng.normal(size=(new, 2, D))).astype(np.float16 if dt == "f16" else np.float32)
    check(mnb, geo, cache, float(vs.max()) * 15, table, [n], [0, new], q, D ** -0.5)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_hidden_keys_do_not_touch_a_row(mnb, new):
    """NaN and infinite scales at the last keys: the rows that see them are NaN, the rows before are as without."""
    t = G.torch()
    rng = np.random.default_rng(933)
    n = 75
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(2, 1, 128, 128, 32, pages)
    cache, vmax = make_cache(rng, geo, table, [n])
    q = rng.normal(size=(new, 2, 128)).astype(np.float16)
    clean, _ = attend(mnb, geo, cache, table, [n], [0, new], q, 0.1)
    for is_v in (False, True):
        for word in (0x00087E00, 0x00087C00):          # NaN, infinity
            dirty = cache.copy()
            base = geo.base(int(table[0, 2]), 0, (n - 1) % 32) + 32 * 128 + (128 if is_v else 0) + 4 * ((n - 1) % 32)
            dirty[base:base + 4] = np.array([word], "<u4").view(np.uint8)
            got, _ = attend(mnb, geo, dirty, table, [n], [0, new], q, 0.1)
            assert t.equal(got[:-1], clean[:-1])
            # (c - z) times an infinite key scale may be a logit of -infinity, which weighs nothing
            assert not t.isfinite(got[-1]).all() or (word == 0x00087C00 and not is_v)
    # a NaN in one query's row stays in that row
    bad = q.copy()
    bad[0, 1, 5] = np.nan
    got = G.host(attend(mnb, geo, cache, table, [n], [0, new], bad, 0.1)[0])
    want = G.host(clean)
    assert np.isnan(got[0, 1]).all() and (got[0, 0] == want[0, 0]).all() and (got[1:] == want[1:]).all()


def test_large_and_small_fp32_queries(mnb):
    rng = np.random.default_rng(934)
    n = 100
    table, pages = sequences(rng, [n], 64)
    geo = o.Geometry(4, 2, 64, 64, 64, pages)
    cache, vmax = make_cache(rng, geo, table, [n], k_scale=1e-3)
    q = rng.normal(size=(3, 4, 64)).astype(np.float32)
    q *= np.array([1e-6, 1.0, 3e5], np.float32)[:, None, None]
    q[1, 0] = 0
    check(mnb, geo, cache, vmax, table, [n], [0, 3], q, 0.05)


def test_strided_queries_and_no_lse(mnb):
    t = G.torch()
    rng = np.random.default_rng(935)
    lens = [90, 41]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(4, 2, 128, 128, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    wide = rng.normal(size=(7, 4 * 128 + 129)).astype(np.float16)
    q = np.ascontiguousarray(wide[:, 1:513]).reshape(7, 4, 128)
    a, _ = attend(mnb, geo, cache, table, lens, [0, 4, 7], q, 0.1)
    b, _ = attend(mnb, geo, cache, table, lens, [0, 4, 7], dev(wide)[:, 1:513].unflatten(1, (4, 128)), 0.1, want_lse=False)
    assert t.equal(a, b)


def test_bounds_larger_than_the_batch(mnb):
    """max_q and max_kv far above the batch's own give the same sums, cut differently; repeated calls the same bits."""
    t = G.torch()
    rng = np.random.default_rng(936)
    lens = [300, 17, 129]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(8, 2, 128, 64, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q = rng.normal(size=(6, 8, 128)).astype(np.float16)
    for max_q, max_kv in ((2, 300), (2, 20000), (50, 301), (300, 9999)):
        a = check(mnb, geo, cache, vmax, table, lens, [0, 2, 4, 6], q, 0.09, max_q=max_q, max_kv=max_kv)
        b, _ = attend(mnb, geo, cache, table, lens, [0, 2, 4, 6], q, 0.09, max_q=max_q, max_kv=max_kv)
        assert t.equal(a, b)


def test_keys_past_the_bound_are_not_seen(mnb):
    rng = np.random.default_rng(937)
    lens = [200]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(2, 1, 64, 64, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q = rng.normal(size=(2, 2, 64)).astype(np.float16)
    check(mnb, geo, cache, vmax, table, lens, [0, 2], q, 0.1, max_kv=77)


@pytest.mark.parametrize("max_q", [1, 3, 40])
def test_tokens_past_the_bound_are_not_written(mnb, max_q):
    """More new tokens than max_q: the first max_q of each sequence as they would be, the rest untouched."""
    rng = np.random.default_rng(940)
    lens, new = [90, 61], [50, 2]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(2, 1, 64, 64, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q = rng.normal(size=(52, 2, 64)).astype(np.float16)
    out, _ = attend(mnb, geo, cache, table, lens, [0, 50, 52], q, 0.1, max_q=max_q)
    w, _, size, reach = o.attention(geo, cache, table, lens, [0, 50, 52], q, 0.1)
    tol = o.attention_tolerance(size, reach, 90, 64, True, vmax)
    got = G.host(out)
    for t in range(52):
        if t - (0 if t < 50 else 50) < max_q:
            assert (np.abs(got[t] - w[t]) <= tol[t]).all(), t
        else:
            assert (got[t] == 7.0).all(), t


def test_device_values_out_of_range_stay_inside(mnb):
    """Lengths past the table, pages outside the cache, offsets past the rows: finite memory use, no fault."""
    t = G.torch()
    rng = np.random.default_rng(938)
    geo = o.Geometry(2, 1, 64, 64, 32, 3)
    cache = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    table = np.array([[0, 1 << 30, -7], [2, 1, 0]], np.int32)
    q = rng.normal(size=(4, 2, 64)).astype(np.float16)
    for lens, q_start in (([96, 1 << 30], [0, 2, 4]), ([-5, 50], [0, 2, 9]), ([40, 40], [-3, 1, 4])):
        d = desc_of(mnb, geo)
        ws = t.empty(1 << 22, dtype=t.uint8, device="cuda")
        out = t.zeros((4, 2, 64), dtype=t.float16, device="cuda")
        mnb.mnb_attention_kv4(d, dev(cache), dev(q), dev(table), dev(np.array(lens, np.int32)),
                              dev(np.array(q_start, np.int32)), 2, 200, out, 0.1, workspace=ws)
        t.cuda.synchronize()
        assert out.shape == (4, 2, 64)


def test_a_captured_graph_and_another_stream(mnb):
    """Norm, append and attention on a side stream and replayed from a graph: the eager calls' bits."""
    t = G.torch()
    rng = np.random.default_rng(939)
    lens = [130, 1000]
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(4, 2, 128, 128, 64, pages)
    cache0, _ = make_cache(rng, geo, table, lens)
    d = desc_of(mnb, geo)
    cache = dev(cache0)
    x = dev(rng.normal(size=(2, 1024)).astype(np.float16))
    w = dev(rng.normal(size=1024).astype(np.float16))
    seq = (dev(table), dev(np.array(lens, np.int32)), dev(np.array([0, 1, 2], np.int32)))
    ang = rng.uniform(0, 6, (1000, 64))
    cos, sin = dev(np.cos(ang).astype(np.float32)), dev(np.sin(ang).astype(np.float32))
    y = t.empty((2, 1024), dtype=t.float16, device="cuda")
    q_out, out = (t.empty((2, 4, 128), dtype=t.float16, device="cuda") for _ in range(2))
    ko = t.empty((2, 2, 128), dtype=t.float16, device="cuda")
    n = mnb.mnb_attention_kv4_workspace_bytes(d, 2, 2, 1, 20000)      # a bound that cuts the keys into splits
    assert n > 0
    ws = t.empty(n, dtype=t.uint8, device="cuda")
    qkv = y.view(2, 8, 128)
    t.cuda.synchronize()

    def issue(stream):
        mnb.mnb_rms_norm(x, w, y, 1e-5, stream=stream)
        mnb.mnb_kv4_append(d, cache, qkv[:, 4:6], qkv[:, 6:], *seq, cos=cos, sin=sin, rotary_dim=128, q=qkv[:, :4],
                           q_out=q_out, stream=stream)
        mnb.mnb_kv4_read(d, cache, *seq, k_out=ko, stream=stream)
        mnb.mnb_attention_kv4(d, cache, q_out, *seq, 1, 20000, out, 0.09, workspace=ws, stream=stream)

    outs = (y, q_out, ko, out, cache)
    issue(t.cuda.current_stream())
    t.cuda.synchronize()
    eager = [v.clone() for v in outs]
    s = t.cuda.Stream()
    for v in outs[:4]:
        v.fill_(float("nan"))
    t.cuda.synchronize()
    issue(s)
    s.synchronize()
    assert all(t.equal(a, b) for a, b in zip(eager, outs))
    s.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            issue(s)
    t.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for v in outs[:4]:
            v.fill_(float("nan"))
        cache.copy_(dev(cache0))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(eager, outs))


def test_binding_refuses_wrong_tensors(mnb):
    t = G.torch()
    geo = o.Geometry(2, 1, 64, 64, 32, 2)
    d = desc_of(mnb, geo)
    cache = t.zeros(geo.bytes, dtype=t.uint8, device="cuda")
    q = t.zeros((1, 2, 64), dtype=t.float16, device="cuda")
    table, kl, qs = (t.zeros(s, dtype=t.int32, device="cuda") for s in ((1, 2), (1,), (2,)))
    for bad in (dict(cache=cache[:-256]), dict(q=q[:, :1]), dict(table=table.long()), dict(kl=kl.repeat(2)),
                dict(qs=qs[:1]), dict(out=q.float())):
        a = dict(cache=cache, q=q, table=table, kl=kl, qs=qs, out=t.empty_like(q))
        a.update(bad)
        with pytest.raises(ValueError):
            mnb.mnb_attention_kv4(d, a["cache"], a["q"], a["table"], a["kl"], a["qs"], 1, 10, a["out"], 0.1)
