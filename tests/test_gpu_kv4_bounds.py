"""Lengths, offsets, pages and windows of any value: the attention stays inside the arrays that the call describes."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import desc_of, dev, sequences
from tests.test_gpu_kv4_attention import attend, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new,max_kv", [(1, 100), (1, 5000), (40, 100), (40, 5000)])
def test_a_cache_without_pages_holds_no_keys(mnb, new, max_kv, dt):
    """Rows of zeros and lse -infinity, whatever the lengths say."""
    rng = np.random.default_rng(980)
    geo = o.Geometry(2, 1, 64, 64, 32, 0)
    table = np.zeros((2, 4), np.int32)
    q = rng.normal(size=(2 * new, 2, 64)).astype(np.float16 if dt == "f16" else np.float32)
    out, lse = attend(mnb, geo, np.zeros(256, np.uint8), table, [60, 90], [0, new, 2 * new], q, 0.1, max_kv=max_kv)
    assert (G.host(out) == 0).all() and np.isneginf(G.host(lse)).all()


@pytest.mark.parametrize("new,max_kv", [(2, 120), (2, 5000), (40, 120), (40, 5000)])
@pytest.mark.parametrize("rest", [[(1 << 31) - 1, -(1 << 31)], [-(1 << 31), -(1 << 31)], [(1 << 31) - 1, -7],
                                  [(1 << 31) - 1, (1 << 31) - 1]])
def test_offsets_of_any_value_stay_inside(mnb, rest, new, max_kv):
    """Offsets that decrease or lie far outside the rows: the sequence before them is as it should be, and rows of no
    sequence and what lies about the outputs stay as they were."""
    t = G.torch()
    rng = np.random.default_rng(981)
    lens = [100, 120, 60]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(4, 2, 128, 64, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    T = new + 3
    q = rng.normal(size=(T, 4, 128)).astype(np.float16)
    start = np.array([0, new] + rest, np.int64)
    d = desc_of(mnb, geo)
    n = mnb.mnb_attention_kv4_workspace_bytes(d, 3, T, new, max_kv)
    ws = t.empty(max(n, 16), dtype=t.uint8, device="cuda")
    buf = t.full((3, T, 4, 128), 7.0, dtype=t.float16, device="cuda")
    mnb.mnb_attention_kv4(d, dev(cache), dev(q), dev(table), dev(np.array(lens, np.int32)), dev(start.astype(np.int32)), new,
                          max_kv, buf[1], 0.1, workspace=ws, workspace_bytes=n)
    w, _, size, reach = o.attention(geo, cache, table, lens[:1], [0, new], q, 0.1)
    got = G.host(buf)
    assert (np.abs(got[1, :new] - w[:new]) <= o.attention_tolerance(size, reach, 120, 128, True, vmax)[:new]).all()
    assert (got[[0, 2]] == 7.0).all()
    if rest[0] < 0:                                    # no offsets past the first sequence lead to a row
        assert (got[1, new:] == 7.0).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 5, (1 << 31) + 7, 1 << 62])
@pytest.mark.parametrize("new", [6, 20, 50])
def test_a_window_wider_than_any_sequence(mnb, new, window, dt):
    """New tokens before position 0 beside ones that see keys: the same bits as without a window."""
    t = G.torch()
    rng = np.random.default_rng((973, new))
    lens = [5, 120]
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(2, 1, 128, 128, 32, pages)
    cache, _ = make_cache(rng, geo, table, lens)
    q = rng.normal(size=(new + 3, 2, 128)).astype(np.float16 if dt == "f16" else np.float32)
    q_start = [0, new, new + 3]
    a, la = attend(mnb, geo, cache, table, lens, q_start, q, 0.1)
    b, lb = attend(mnb, geo, cache, table, lens, q_start, q, 0.1, window=window)
    assert t.equal(a, b) and t.equal(la, lb)
    assert a[new - 1].any() and not a[0].any()
