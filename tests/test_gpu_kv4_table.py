"""The page table as the binding takes it."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import desc_of, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def test_columns_of_a_wider_table_are_refused(mnb):
    """Their rows' pitch would be taken for the rows' length: entries beside the slice, and past the last row's end."""
    t = G.torch()
    geo = o.Geometry(2, 1, 64, 64, 32, 16)
    full = dev(np.arange(32, dtype=np.int32).reshape(2, 16) % 16)
    cache = t.full((geo.bytes,), 0x5A, dtype=t.uint8, device="cuda")
    k, q = (t.ones((2, h, 64), dtype=t.float16, device="cuda") for h in (1, 2))
    ko, out = t.empty_like(k), t.empty_like(q)
    lens, start = dev(np.array([200, 200], np.int32)), dev(np.array([0, 1, 2], np.int32))
    d = desc_of(mnb, geo)
    for table in (full[:, 12:16], full[:, :4], full.t()[:2], full[:, ::2]):
        with pytest.raises(ValueError, match="block_table"):
            mnb.mnb_kv4_append(d, cache, k, k, table, lens, start)
        with pytest.raises(ValueError, match="block_table"):
            mnb.mnb_kv4_read(d, cache, table, lens, start, ko)
        with pytest.raises(ValueError, match="block_table"):
            mnb.mnb_attention_kv4(d, cache, q, table, lens, start, 1, 200, out, 0.1)
    assert bool((cache == 0x5A).all())


def test_one_row_of_a_wider_table_and_its_length(mnb):
    """A slice of one row is dense: tokens past its length have no place, whatever the wider table says there."""
    t = G.torch()
    rng = np.random.default_rng(990)
    geo = o.Geometry(2, 1, 64, 64, 32, 16)
    full = dev(rng.permutation(16).astype(np.int32).reshape(1, 16))
    part = full[:, 12:14]                              # 64 tokens
    k, v = (rng.normal(size=(10, 1, 64)).astype(np.float16) for _ in range(2))
    want = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    cache = dev(want)
    table = part.cpu().numpy()
    o.append(geo, want, table, [69], [0, 10], k, v)    # positions 59..68
    seq = (part, dev(np.array([69], np.int32)), dev(np.array([0, 10], np.int32)))
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), *seq)
    assert (cache.cpu().numpy() == want).all()
    vo = t.full((10, 1, 64), 9.0, dtype=t.float16, device="cuda")
    mnb.mnb_kv4_read(desc_of(mnb, geo), cache, *seq, v_out=vo)
    got = vo.cpu().numpy()
    V = o.gather(geo, want, table[0], 0, 64)[1]
    assert (got[:5, 0] == V[59:].astype(np.float16)).all() and (got[5:] == 0).all()
