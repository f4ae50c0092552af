"""Attention through a window beside which the first tokens stay visible, on the GPU against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import desc_of, dev, sequences
from tests.test_gpu_kv4_attention import CASES, attend as attend_causal, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def attend(mnb, geo, cache, table, lens, q_start, q, scale, window, sinks, max_q=None, max_kv=None, stream=None):
    t = G.torch()
    d = desc_of(mnb, geo)
    dq = dev(q) if isinstance(q, np.ndarray) else q
    T = dq.shape[0]
    max_q = int(np.diff(q_start).max()) if max_q is None else max_q
    max_kv = int(max(lens)) if max_kv is None else max_kv
    n = mnb.mnb_attention_kv4_sinks_workspace_bytes(d, len(lens), T, max_q, max_kv, window, sinks)
    ws = t.full((max(n, 256),), 0xFF, dtype=t.uint8, device="cuda")      # NaN to whatever reads it unwritten
    out = t.full(tuple(dq.shape), 7.0, dtype=dq.dtype, device="cuda")
    lse = t.full(tuple(dq.shape[:2]), 7.0, device="cuda")
    mnb.mnb_attention_kv4_sinks(d, dev(cache) if isinstance(cache, np.ndarray) else cache, dq, dev(table),
                                dev(np.array(lens, np.int32)), dev(np.array(q_start, np.int32)), max_q, max_kv, out,
                                scale, window, sinks, lse=lse, workspace=ws, workspace_bytes=n, stream=stream)
    return out, lse


def check(mnb, geo, cache, vmax, table, lens, q_start, q, scale, window, sinks, max_kv=None, seen_by=None, **kw):
    """seen_by: the table that the call gets, where it differs from the oracle's in pages that no row sees."""
    out, lse = attend(mnb, geo, cache, table if seen_by is None else seen_by, lens, q_start, q, scale, window, sinks,
                      max_kv=max_kv, **kw)
    w, wl, size, reach = o.attention(geo, cache, table, lens, q_start, q, scale, True, window, max_kv, sinks)
    keys = max(max(lens), 1)
    tol = o.attention_tolerance(size, reach, keys, geo.D, q.dtype == np.float16, vmax)
    err = np.abs(G.host(out) - w)
    assert np.isfinite(G.host(out)).all()
    assert (err <= tol).all(), "worst %.3g of the bound" % float((err / tol).max())
    gl = G.host(lse)
    empty = np.isneginf(wl)
    assert (np.isneginf(gl) == empty).all() and (G.host(out)[empty] == 0).all()
    lt = o.lse_tolerance(np.where(empty, 0, wl), reach, keys, geo.D)
    assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, wl)) <= lt).all()
    return out, lse


def kind(dt):
    return np.float16 if dt == "f16" else np.float32


def unseen(rng, table, lens, new, window, sinks, page):
    """The table with every page that no row sees turned into something else: -1, a page of another, garbage."""
    t = table.copy()
    for b, (n, m) in enumerate(zip(lens, new)):
        j = np.arange(max(n, 1))
        seen = (j < sinks) | (j > n - m - window) if window else j >= 0
        for p in range(-(-n // page)):
            if m == 0 or not seen[p * page:(p + 1) * page].any():
                t[b, p] = rng.choice([-1, 0, 1 << 30])
    return t


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("window,sinks", [(37, 4), (1, 1), (20, 33), (70, 0), (64, 1000)])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:5] + (c[5][0], c[6][0]))) for c in CASES])
def test_against_the_oracle(mnb, case, window, sinks, dt):
    D, group, page, H, Hkv, new, lens = case
    rng = np.random.default_rng((950, D, group, page, H, lens[0], window))
    table, pages = sequences(rng, lens, page)
    geo = o.Geometry(H, Hkv, D, group, page, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (1.5 * rng.normal(size=(q_start[-1], H, D))).astype(kind(dt))
    check(mnb, geo, cache, vmax, table, lens, q_start, q, D ** -0.5, window, sinks,
          seen_by=unseen(rng, table, lens, new, window, sinks, page))


LONG = [  # D, group, q heads, kv heads, new tokens, cached with them, window, sinks
    (128, 128, 4, 1, [1, 1], [3000, 300], 500, 4),        # one workgroup a row set
    (128, 128, 4, 2, [1, 1], [4100, 1500], 1500, 40),     # splits
    (64, 64, 2, 1, [3], [4900], 2600, 700),               # sinks over several splits
    (256, 64, 4, 1, [1, 2, 0], [5100, 33, 0], 1300, 65),
    (128, 64, 3, 1, [40, 2], [2300, 700], 900, 4),        # many rows
    (64, 32, 2, 1, [35], [4500], 2000, 33),
    (256, 128, 2, 1, [20], [4400], 700, 1500),
    (128, 128, 8, 4, [300, 3], [1100, 1099], 130, 5),     # a gap in most row sets, none in the first
    (128, 128, 1, 1, [700], [700], 50, 3),                # a prompt longer than its window
    (64, 64, 4, 2, [260], [400], 33, 100),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", LONG, ids=["-".join(map(str, c[:4] + (c[4][0], c[5][0]) + c[6:])) for c in LONG])
def test_long_sequences(mnb, case, dt):
    D, group, H, Hkv, new, lens, window, sinks = case
    rng = np.random.default_rng((951, D, H, lens[0]))
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(H, Hkv, D, group, 64, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (1.5 * rng.normal(size=(q_start[-1], H, D))).astype(kind(dt))
    check(mnb, geo, cache, vmax, table, lens, q_start, q, D ** -0.5, window, sinks,
          seen_by=unseen(rng, table, lens, new, window, sinks, 64))


@pytest.mark.parametrize("new", [1, 5, 40])
def test_what_the_gap_holds_does_not_touch_a_row(mnb, new):
    """NaN and infinite scales in every hidden place: the rows' bits stay."""
    t = G.torch()
    rng = np.random.default_rng(952)
    n, window, sinks = 900, 200, 10
    table, pages = sequences(rng, [n], 32)
    geo = o.Geometry(2, 1, 128, 64, 32, pages)
    cache, _ = make_cache(rng, geo, table, [n])
    q = rng.normal(size=(new, 2, 128)).astype(np.float16)
    clean = attend(mnb, geo, cache, table, [n], [0, new], q, 0.1, window, sinks)
    blocks = cache.reshape(-1, geo.B)
    for p in range(sinks, n - new - window + 1):
        words = blocks[int(table[0, p // 32]), 32 * 128:].view("<u4").reshape(2, 32, 2)
        words[:, p % 32] = rng.choice(np.array([0x00087E00, 0x00087C00, 0x0008FC00], np.uint32), (2, 2))
    dirty = attend(mnb, geo, cache, table, [n], [0, new], q, 0.1, window, sinks)
    assert t.equal(clean[0], dirty[0]) and t.equal(clean[1], dirty[1])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_no_window_is_the_causal_attention(mnb, dt):
    """Window 0, and one that no position passes, whatever the sinks: mnb_attention_kv4's bits."""
    t = G.torch()
    rng = np.random.default_rng(953)
    lens, new = [300, 1200, 40], [2, 33, 1]
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(4, 2, 128, 128, 64, pages)
    cache, _ = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = rng.normal(size=(36, 4, 128)).astype(kind(dt))
    want = attend_causal(mnb, geo, cache, table, lens, q_start, q, 0.1)
    for window, sinks in ((0, 4), (0, 0), (1200, 7), (1 << 40, 1 << 40)):
        got = attend(mnb, geo, cache, table, lens, q_start, q, 0.1, window, sinks)
        assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_rows_that_see_nothing(mnb, dt):
    """Empty sequences, new tokens before position 0, and bounds far above the batch's own."""
    rng = np.random.default_rng(954)
    lens, new = [0, 5, 140, 0], [2, 9, 3, 0]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(4, 2, 128, 128, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = rng.normal(size=(14, 4, 128)).astype(kind(dt))
    for window, sinks in ((3, 2), (50, 40)):
        check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, window, sinks)
        check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, window, sinks, max_kv=5000)
        check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, window, sinks, max_kv=100)
        check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.1, window, sinks, max_q=300, max_kv=90000)


def test_a_part_of_a_batch_writes_its_rows_alone(mnb):
    rng = np.random.default_rng(955)
    lens = [400, 350]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(2, 1, 64, 64, 32, pages)
    cache, _ = make_cache(rng, geo, table, lens)
    q = rng.normal(size=(12, 2, 64)).astype(np.float16)
    whole, _ = attend(mnb, geo, cache, table, lens, [0, 7, 12], q, 0.1, 100, 4)
    part, lse = attend(mnb, geo, cache, table[1:], lens[1:], [7, 11], q, 0.1, 100, 4)
    got = G.host(part)
    assert (got[:7] == 7.0).all() and (got[11:] == 7.0).all() and (G.host(lse)[:7] == 7.0).all()
    w, _, size, reach = o.attention(geo, cache, table[1:], lens[1:], [7, 11], q, 0.1, True, 100, None, 4)
    # 4 new tokens instead of 5: their positions are one further
    tol = o.attention_tolerance(size, reach, 400, 64, True, 15)
    assert (np.abs(got - w)[7:11] <= tol[7:11]).all()


def test_replays_and_streams_give_the_eager_bits(mnb):
    t = G.torch()
    rng = np.random.default_rng(956)
    lens = [1300, 5000]
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(4, 2, 128, 128, 64, pages)
    cache, d = make_cache(rng, geo, table, lens)[0], None
    cache, d = dev(cache), desc_of(mnb, geo)
    q = dev(rng.normal(size=(3, 4, 128)).astype(np.float16))
    seq = (dev(table), dev(np.array(lens, np.int32)), dev(np.array([0, 2, 3], np.int32)))
    n = mnb.mnb_attention_kv4_sinks_workspace_bytes(d, 2, 3, 2, 5000, 2000, 40)
    assert n > 0
    ws, out = t.empty(n, dtype=t.uint8, device="cuda"), t.empty_like(q)

    def issue(stream):
        mnb.mnb_attention_kv4_sinks(d, cache, q, *seq, 2, 5000, out, 0.09, 2000, 40, workspace=ws, stream=stream)

    issue(t.cuda.current_stream())
    t.cuda.synchronize()
    eager = out.clone()
    s = t.cuda.Stream()
    out.fill_(float("nan"))
    s.wait_stream(t.cuda.current_stream())
    issue(s)
    s.synchronize()
    assert t.equal(eager, out)
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            issue(s)
    t.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(eager, out)
