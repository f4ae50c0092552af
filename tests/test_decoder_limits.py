"""Limits of the calls between the products, through the C ABI and the binding.  No GPU: every check runs on the
host before any HIP call."""
import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import INVALID, P, _refused, append, attend, desc, read


def test_a_cache_whose_size_overflows_is_refused_by_every_call():
    big = desc(q_heads=65536, kv_heads=65536, head_dim=256, group_size=32, page_size=256, num_pages=(1 << 31) - 1)
    row = 65536 * 256
    _refused(INVALID, append, d=big, q_s=row, k_s=row, v_s=row, rot=64)
    _refused(INVALID, read, d=big)
    _refused(INVALID, attend, d=big, q_s=row)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_kv4_cache_bytes(big)
    assert mnb.mnb_attention_kv4_workspace_bytes(big, 1, 1, 1, 100) == 0 and "overflow" in mnb.mnb_last_error()


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_a_scale_that_overflows_in_the_units_of_log2_is_refused(scale):
    _refused(INVALID, attend, scale=scale)
