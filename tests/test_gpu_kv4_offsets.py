"""Rows of the new tokens' arrays that belong to no sequence: the first sequence need not start at row 0."""
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


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("q_start,lens,rows", [
    ([4, 8, 12], [20, 30], 12),                       # a part of a batch, by its offsets in the whole arrays
    ([3, 5], [10], 5),
    ([3, 3, 3, 5, 5], [40, 7, 35, 9], 9),             # empty sequences about it, rows past the last
    ([600, 601, 640], [33, 70], 700),                 # whole runs of rows before the first
])
def test_rows_before_the_first_sequence_have_no_place(mnb, q_start, lens, rows, dt):
    """They are not stored and read as zeros; their queries are turned by position 0."""
    t = G.torch()
    rng = np.random.default_rng((950, rows, len(lens)))
    H, Hkv, D = 4, 2, 64
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(H, Hkv, D, 32, 32, pages)
    kind = np.float16 if dt == "f16" else np.float32
    q, k, v = (rng.normal(size=(rows, h, D)).astype(kind) for h in (H, Hkv, Hkv))
    ang = rng.uniform(0.1, 6.2, (max(lens), D // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    want = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    cache = dev(want)
    pos = o.append(geo, want, table, lens, q_start, k, v, cos, sin, D)
    assert (pos[:q_start[0]] == -1).all() and (pos[q_start[-1]:] == -1).all()
    q_out = t.full((rows, H, D), 9.0, dtype=dev(q).dtype, device="cuda")
    seq = (dev(table), dev(np.array(lens, np.int32)), dev(np.array(q_start, np.int32)))
    mnb.mnb_kv4_append(desc_of(mnb, geo), cache, dev(k), dev(v), *seq, cos=dev(cos), sin=dev(sin), rotary_dim=D,
                       q=dev(q), q_out=q_out)
    got = cache.cpu().numpy()
    assert (got == want).all(), "%d bytes differ" % (got != want).sum()
    assert (q_out.cpu().numpy() == o.rotate(q, pos, cos, sin, D).astype(kind)).all()

    ko, vo = (t.full((rows, Hkv, D), 9.0, dtype=dev(q).dtype, device="cuda") for _ in range(2))
    mnb.mnb_kv4_read(desc_of(mnb, geo), cache, *seq, ko, vo)
    ko, vo = ko.cpu().numpy(), vo.cpu().numpy()
    for b in range(len(lens)):
        for h in range(Hkv):
            K, V = o.gather(geo, want, table[b], h, lens[b])
            at = slice(q_start[b], q_start[b + 1])
            n = q_start[b + 1] - q_start[b]
            assert (ko[at, h] == K[lens[b] - n:].astype(kind)).all() and (vo[at, h] == V[lens[b] - n:].astype(kind)).all()
    for out in (ko, vo):
        assert (out[:q_start[0]] == 0).all() and (out[q_start[-1]:] == 0).all()
