"""Low-rank adapters of many requests on the GPU against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import requests as o
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def kind(dt):
    return np.float16 if dt == "f16" else np.float32


def operands(rng, m, k, n, rank, count, dt, mixed=False):
    a = (rng.normal(size=(count, rank, k)) * k ** -0.5).astype(kind(dt))
    b = (rng.normal(size=(count, n, rank)) * rank ** -0.5).astype(kind(dt))
    x = rng.normal(size=(m, k)).astype(kind(dt))
    base = rng.normal(size=(m, n)).astype(kind(dt))
    scales = rng.uniform(0.25, 2, count).astype(np.float32)
    ranks = rng.integers(-1, rank + 3, count).astype(np.int32) if mixed else None
    if mixed:                          # what lies behind an adapter's rank is not read
        for g in range(count):
            a[g, max(0, ranks[g]):] = np.nan
            b[g, :, max(0, ranks[g]):] = np.inf
    return a, b, x, base, scales, ranks


def run(mnb, a, b, scales, ranks, adapter, x, base, stream=None, **kw):
    t = G.torch()
    dev = {k: None if v is None else G.to_dev(v) for k, v in
           dict(a=a, b=b, scales=scales, ranks=ranks, adapter=adapter.astype(np.int32), x=x, base=base).items()}
    d = mnb.adapter_desc(b.shape[1], a.shape[2], a.shape[1], a.shape[0], dev["x"].dtype)
    size = mnb.mnb_adapters_workspace_bytes(d, x.shape[0])
    ws = t.full((max(size, 256),), 0xFF, dtype=t.uint8, device="cuda")   # NaN to whatever reads it unwritten
    y = t.full((x.shape[0], b.shape[1]), 7.0, dtype=dev["x"].dtype, device="cuda")
    mnb.mnb_adapters_add(d, dev["a"], dev["b"], dev["scales"], dev["adapter"], dev["x"], y, base=dev["base"],
                         ranks=dev["ranks"], workspace=ws, workspace_bytes=size, stream=stream, **kw)
    return y


def check(mnb, a, b, scales, ranks, adapter, x, base):
    y = run(mnb, a, b, scales, ranks, adapter, x, base)
    w, tol = o.adapters(a, b, scales, ranks, adapter, x, base)
    G.assert_within(G.host(y), w, None, "adapters", bound=tol)
    return y


SIZES = [  # m, k, n, rank, count
    (1, 64, 64, 16, 1), (1, 1, 1, 1, 1), (1, 4096, 300, 8, 3), (2, 65, 63, 7, 2), (5, 130, 65, 17, 9),
    (15, 512, 128, 32, 4), (16, 521, 5, 33, 40), (17, 63, 257, 64, 2), (33, 1000, 130, 9, 33), (50, 257, 64, 100, 3),
    (100, 2050, 70, 12, 7), (64, 256, 40, 128, 5), (130, 96, 513, 4, 130), (300, 40, 90, 16, 300), (7, 7, 1000, 2, 5),
    (1030, 200, 321, 24, 6), (2049, 72, 50, 3, 3), (4100, 136, 77, 20, 5), (4113, 70, 66, 65, 2),
    # two launches: many sets of rows and adapters, or ranks past 64
    (800, 130, 70, 16, 200), (1030, 200, 321, 24, 40), (1000, 513, 65, 33, 64), (830, 2100, 40, 9, 64), (70, 300, 60, 100, 9),
    (3, 5000, 200, 128, 3), (2100, 64, 300, 8, 5), (33, 600, 16400, 5, 33),
    # several blocks of columns a workgroup, the last one's missing
    (130, 64, 32800, 40, 6), (600, 72, 8200, 128, 3), (50, 100, 66000, 64, 20),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("order", ["grouped", "any", "mixed"])
@pytest.mark.parametrize("size", SIZES, ids=["-".join(map(str, s)) for s in SIZES])
def test_against_the_oracle(mnb, size, order, dt):
    m, k, n, rank, count = size
    rng = np.random.default_rng((970, m, k, n, rank))
    a, b, x, base, scales, ranks = operands(rng, m, k, n, rank, count, dt, order == "mixed")
    adapter = rng.integers(-1, count + 1, m)           # some rows without: -1 and the first index behind
    if order == "grouped":
        adapter = np.sort(adapter)
    check(mnb, a, b, scales, ranks, adapter, x, base)


@pytest.mark.parametrize("size", [(8193, 8193, "f16"), (4097, 8193, "f32")])
def test_base_and_output_past_the_caches(mnb, size):
    m, n, dt = size
    rng = np.random.default_rng((969, m))
    a, b, x, base, scales, _ = operands(rng, m, 24, n, 3, 4, dt)
    adapter = rng.integers(-1, 4, m)
    got = G.host(run(mnb, a, b, scales, None, adapter, x, base))
    for i in range(0, m, 1000):                        # the definition, some rows at a time
        rows = slice(i, i + 1000)
        w, tol = o.adapters(a, b, scales, None, adapter[rows], x[rows], base[rows])
        G.assert_within(got[rows], w, None, "adapters", bound=tol)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m", [3, 1100, 9000])
def test_without_base_scales_or_adapters(mnb, m, dt):
    rng = np.random.default_rng(971)
    a, b, x, base, _, _ = operands(rng, m, 100, 70, 10, 4, dt)
    adapter = rng.integers(-1, 4, m)
    check(mnb, a, b, None, None, adapter, x, None)
    got = G.host(run(mnb, a, b, None, None, np.full(m, -1), x, None))
    assert (got == 0).all()
    got = G.host(run(mnb, a, b, None, None, np.full(m, 1 << 30), x, base))
    assert (got == base.astype(np.float64)).all()
    none = a[:0], b[:0]
    assert (G.host(run(mnb, *none, None, None, adapter, x, base)) == base.astype(np.float64)).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m", [5, 1040, 9001])
def test_slices_of_wider_rows_and_in_place(mnb, m, dt):
    """x, base and y as columns of wider rows at an odd element; what is beside them stays; y may be base."""
    t = G.torch()
    rng = np.random.default_rng(972)
    k, n = 130, 77
    a, b, x, base, scales, _ = operands(rng, m, k, n, 16, 3, dt)
    adapter = rng.integers(-1, 3, m)
    want = run(mnb, a, b, scales, None, adapter, x, base)
    wx, wb, wy = (t.full((m, w), 3.0, dtype=want.dtype, device="cuda") for w in (k + 9, n + 5, n + 12))
    wx[:, 3:3 + k], wb[:, 5:] = G.to_dev(x), G.to_dev(base)
    d = mnb.adapter_desc(n, k, 16, 3, want.dtype)
    ws = t.empty(mnb.mnb_adapters_workspace_bytes(d, m), dtype=t.uint8, device="cuda")
    ops = (d, G.to_dev(a), G.to_dev(b), G.to_dev(scales), G.to_dev(adapter.astype(np.int32)), wx[:, 3:3 + k])
    y = wy[:, 1:1 + n]
    mnb.mnb_adapters_add(*ops, y, base=wb[:, 5:], workspace=ws)
    assert t.equal(y, want) and (wy[:, :1] == 3).all() and (wy[:, 1 + n:] == 3).all()
    mnb.mnb_adapters_add(*ops, wb[:, 5:], base=wb[:, 5:], workspace=ws)
    assert t.equal(wb[:, 5:], want) and (wb[:, :5] == 3).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m", [20, 1050, 9010])
def test_bad_values_stay_in_their_row(mnb, m, dt):
    """NaN and infinity in one row, and in an adapter's slot that no row has: the other rows' bits stay."""
    t = G.torch()
    rng = np.random.default_rng(973)
    a, b, x, base, scales, _ = operands(rng, m, 150, 90, 20, 4, dt)
    adapter = rng.integers(-1, 3, m)
    adapter[7], adapter[8] = 0, -1
    clean = run(mnb, a, b, scales, None, adapter, x, base)
    a[3], b[3] = np.nan, np.inf
    for bad in (np.nan, np.inf, -np.inf):
        dirty = x.copy()
        dirty[7, 5], dirty[8] = bad, bad                # row 8 has no adapter
        got = run(mnb, a, b, scales, None, adapter, dirty, base)
        keep = [i for i in range(m) if i != 7]
        assert t.equal(got[keep], clean[keep]) and not t.isfinite(got[7]).any()


@pytest.mark.parametrize("m,n", [(1, 64), (40, 64), (70, 30000)])
def test_large_and_small_products_between(mnb, m, n):
    """h far past fp16's range, and far below it, while y is inside."""
    rng = np.random.default_rng(974)
    for size, back in ((60000.0, 2.0 ** -20), (2.0 ** -14, 2.0 ** 12)):
        a, b, x, base, _, _ = operands(rng, m, 600, n, 24, 9, "f16")
        x = (x.astype(np.float64) * size / 8).astype(np.float16)
        scales = np.full(9, back, np.float32)
        check(mnb, a, b, scales, None, rng.integers(0, 9, m), x, base)


def test_repeated_calls_graphs_and_streams_give_the_same_bits(mnb):
    """Two calls that share a workspace, one after the other, on a side stream and replayed from a graph."""
    t = G.torch()
    rng = np.random.default_rng(975)
    sets = []
    for m, k, n, rank, dt in ((9, 512, 200, 16, "f16"), (1100, 200, 130, 70, "f16"), (30, 300, 100, 8, "f32"),
                              (9000, 100, 65, 20, "f32")):
        a, b, x, base, scales, _ = operands(rng, m, k, n, rank, 4, dt)
        dev = [G.to_dev(v) for v in (a, b, scales, rng.integers(-1, 4, m).astype(np.int32), x, base)]
        sets.append((mnb.adapter_desc(n, k, rank, 4, dev[4].dtype), dev, t.empty_like(dev[5])))
    ws = t.empty(max(mnb.mnb_adapters_workspace_bytes(d, v[4].shape[0]) for d, v, _ in sets), dtype=t.uint8, device="cuda")

    def issue(stream):
        for d, (a, b, s, which, x, base), y in sets:
            mnb.mnb_adapters_add(d, a, b, s, which, x, y, base=base, workspace=ws, stream=stream)

    issue(t.cuda.current_stream())
    t.cuda.synchronize()
    eager = [y.clone() for _, _, y in sets]
    s = t.cuda.Stream()
    for _, _, y in sets:
        y.fill_(float("nan"))
    s.wait_stream(t.cuda.current_stream())
    issue(s)
    s.synchronize()
    assert all(t.equal(e, y) for e, (_, _, y) in zip(eager, sets))
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            issue(s)
    t.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for _, _, y in sets:
            y.fill_(float("nan"))
        ws.fill_(0xFF)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(e, y) for e, (_, _, y) in zip(eager, sets))


def test_binding_refuses_wrong_tensors(mnb):
    t = G.torch()
    d = mnb.adapter_desc(32, 64, 8, 2, t.float16)
    f = dict(dtype=t.float16, device="cuda")
    good = dict(a=t.zeros(2, 8, 64, **f), b=t.zeros(2, 32, 8, **f), scales=t.zeros(2, device="cuda"),
                adapter=t.zeros(3, dtype=t.int32, device="cuda"), x=t.zeros(3, 64, **f), y=t.zeros(3, 32, **f),
                base=t.zeros(3, 32, **f), ranks=t.zeros(2, dtype=t.int32, device="cuda"),
                workspace=t.zeros(1 << 16, dtype=t.uint8, device="cuda"))
    mnb.mnb_adapters_add(d, **good)
    for name, bad in (("a", good["a"][:1]), ("a", good["a"].float()), ("b", good["b"].transpose(1, 2)), ("x", good["x"][:2]),
                      ("x", good["x"].float()), ("y", good["y"][:, :31]), ("base", good["base"].float()),
                      ("base", good["base"].t()), ("scales", good["scales"].half()), ("scales", good["scales"][:1]),
                      ("ranks", good["ranks"].long()), ("adapter", good["adapter"].long()),
                      ("adapter", good["adapter"][:2]), ("x", good["x"].cpu()), ("adapter", good["adapter"].cpu())):
        with pytest.raises(ValueError):
            mnb.mnb_adapters_add(d, **dict(good, **{name: bad}))
    mnb.mnb_adapters_add(d, **dict(good, workspace=None))            # few rows need none
    a, b = t.zeros(2, 40, 64, **f), t.zeros(2, 32, 40, **f)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_adapters_add(mnb.adapter_desc(32, 64, 40, 2, t.float16), **dict(good, a=a, b=b, workspace=None))


@pytest.mark.parametrize("m,rank,count,name", [(1, 16, 4, "adapters_one"), (60, 32, 30, "adapters_one"), (3, 33, 2, "adapters"),
                                               (5000, 16, 9, "adapters")])
def test_which_kernels_ran(mnb, m, rank, count, name):
    rng = np.random.default_rng(976)
    a, b, x, base, scales, _ = operands(rng, m, 80, 70, rank, count, "f16")
    run(mnb, a, b, scales, None, rng.integers(0, count, m), x, base)
    assert mnb.mnb_last_variant() == name
