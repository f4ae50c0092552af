"""Argument checks of the attention with first tokens that stay visible, through the C ABI.  No GPU."""
import ctypes

import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import F32, INVALID, UNSUPPORTED, DEVICE, P, _no_device, _refused, desc


def attend(d=None, **kw):
    a = dict(cache=P, table=P, ts=4, kl=P, qs=P, batch=2, tokens=5, mq=3, mk=250, dt=mnb.MNB_F16, q=P, q_s=1024, scale=0.1,
             window=100, sinks=4, out=P, lse=None, ws=P, wb=1 << 30)
    a.update(kw)
    d = d or desc()
    return mnb.lib.mnb_attention_kv4_sinks(ctypes.byref(d), a["cache"], a["table"], a["ts"], a["kl"], a["qs"], a["batch"],
                                           a["tokens"], a["mq"], a["mk"], a["dt"], a["q"], a["q_s"], a["scale"],
                                           a["window"], a["sinks"], a["out"], a["lse"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(batch=-1), dict(tokens=-1), dict(mq=-1), dict(mk=-1), dict(window=-1), dict(sinks=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q_s=1023), dict(table=None), dict(kl=None), dict(qs=None),
    dict(ts=0), dict(q=None), dict(out=None), dict(cache=None), dict(cache=P + 16), dict(lse=P + 2), dict(out=P + 1),
    dict(dt=F32, q=P + 2), dict(ws=None), dict(ws=P + 16), dict(wb=16)])
def test_refuses(kw):
    # many keys and few rows: a call that needs its workspace
    _refused(INVALID, attend, mk=kw.pop("mk", 100000), window=kw.pop("window", 50000), **kw)


def test_unsupported():
    _refused(UNSUPPORTED, attend, batch=70000, tokens=70000)
    _refused(UNSUPPORTED, attend, mk=(1 << 30) + 1)
    _refused(UNSUPPORTED, attend, mq=1 << 30)
    _refused(UNSUPPORTED, attend, d=desc(head_dim=96))


def test_empty_requests_are_noops():
    for kw in (dict(tokens=0), dict(batch=0), dict(mq=0)):
        assert attend(**kw) == 0 and mnb.mnb_last_variant() == "noop"


def test_the_workspace_follows_the_window():
    d = desc()
    size = mnb.mnb_attention_kv4_sinks_workspace_bytes
    assert size(d, 1, 1, 1, 100000, 500, 4) == 0                     # one workgroup a row set, whatever the length
    n = size(d, 1, 1, 1, 100000, 30000, 4)
    assert 0 < n == size(d, 1, 1, 1, 1 << 30, 30000, 4)
    assert size(d, 1, 1, 1, 100000, 0, 4) == mnb.mnb_attention_kv4_workspace_bytes(d, 1, 1, 1, 100000)
    assert size(d, 1, 1, 1, 100000, 1 << 62, 1 << 62) == mnb.mnb_attention_kv4_workspace_bytes(d, 1, 1, 1, 100000)
    assert size(d, 0, 0, 0, 0, 1, 1) == 0
    for bad in ((-1, 4), (4, -1)):
        assert size(d, 1, 1, 1, 100, *bad) == 0 and mnb.mnb_last_error() != ""
    args = dict(batch=1, tokens=1, mq=1, mk=100000, window=30000)
    _refused(INVALID, attend, wb=n - 1, **args)
    if _no_device():
        _refused(DEVICE, attend, wb=n, **args)
