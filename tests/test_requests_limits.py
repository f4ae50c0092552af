"""Sizes of the adapters and of the verification at the ends of their ranges, through the C ABI.  No GPU."""
import ctypes

import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import DEVICE, F16, F32, INVALID, _no_device, _refused
from tests.test_requests_abi import add

MOST = (1 << 31) - 1


@pytest.mark.parametrize("dt", [F16, F32])
@pytest.mark.parametrize("kw", [dict(k=1 << 24, xs=1 << 24), dict(n=1 << 24, ys=1 << 24, bs=1 << 24)])
def test_weights_whose_bytes_overflow_are_refused(kw, dt):
    """[count, rank, k] or [count, n, rank] of 2^62 elements."""
    _refused(INVALID, add, rank=128, count=MOST, dt=dt, wb=1 << 40, **kw)
    d = mnb.mnb_adapter_desc(kw.get("n", 96), kw.get("k", 128), 128, MOST, dt, 0)
    assert mnb.lib.mnb_adapters_workspace_bytes(ctypes.byref(d), 5) == 0 and mnb.mnb_last_error() != ""
    if _no_device():
        _refused(DEVICE, add, rank=128, count=1 << 20, dt=dt, wb=1 << 40, **kw)
        _refused(DEVICE, add, count=MOST, dt=dt, wb=1 << 40)
