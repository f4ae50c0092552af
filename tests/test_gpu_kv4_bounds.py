"""Lengths, offsets and pages of any value: the attention stays inside the arrays that the call describes."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import desc_of, dev
from tests.test_gpu_kv4_attention import attend

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
