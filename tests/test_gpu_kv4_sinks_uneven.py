"""A long window over many sequences, one of them long: its keys are cut, the others' rows are of one piece or none."""
import numpy as np
import pytest

from oracle import decoder as o
from tests.test_gpu_kv4 import sequences
from tests.test_gpu_kv4_attention import make_cache
from tests.test_gpu_kv4_sinks import check, kind, mnb, unseen  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("new,window,sinks", [(1, 6000, 4), (3, 5200, 300), (1, 11000, 33)])
def test_one_long_sequence_among_short_ones(mnb, new, window, sinks, dt):  # noqa: F811
    rng = np.random.default_rng((957, window))
    lens = [12000, 0, 1, 40] + [int(v) for v in rng.integers(1, 300, 35)] + [6100]
    rows = [new] * len(lens)
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(8, 8, 64, 64, 64, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(rows)])
    q = (1.5 * rng.normal(size=(q_start[-1], 8, 64))).astype(kind(dt))
    check(mnb, geo, cache, vmax, table, lens, q_start, q, 0.125, window, sinks,
          seen_by=unseen(rng, table, lens, rows, window, sinks, 64))
    assert mnb.mnb_last_variant() == "attention_kv4_sinks_split"
