"""Sizes of the adapters and of the verification at the ends of their ranges, through the C ABI.  No GPU."""
import ctypes
import random

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


def test_a_workspace_for_every_batch_up_to_a_size():
    """The documented bound holds for all smaller batches, whose own sizes may be larger than the largest one's."""
    rng = random.Random(1)
    uneven = 0
    for case in range(300):
        n, k = (int(2 ** rng.uniform(0, 15)) for _ in range(2))
        rank, count, dt = rng.randint(1, 128), int(2 ** rng.uniform(0, 9)), rng.choice([F16, F32])
        if case == 0:
            n, k, rank, count, dt = 4096, 4096, 16, 4, F16
        d = mnb.mnb_adapter_desc(n, k, rank, count, dt, 0)
        pitch = next(p for p in (16, 32, 64, 128) if rank <= p)
        sizes = sorted({int(2 ** rng.uniform(0, 17)) for _ in range(60)} | {8120, 8580})
        need = [mnb.mnb_adapters_workspace_bytes(d, m) for m in sizes]
        for i, m in enumerate(sizes):
            assert max(need[:i + 1]) <= 4 * pitch * min(8 * m, m + 32768), (n, k, rank, m)
        uneven += any(a > b for a, b in zip(need, need[1:]))
    assert uneven > 0
