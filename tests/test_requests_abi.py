"""Argument checks of the adapters and of the verification through the C ABI.  No GPU: every check runs on the host
before any HIP call, and a well-formed request without a device returns MNB_ERR_DEVICE."""
import ctypes

import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import DEVICE, F16, F32, INVALID, UNSUPPORTED, P, _no_device, _refused


def add(**kw):
    a = dict(n=96, k=128, rank=16, count=3, dt=F16, reserved=0, a=P, b=P, sc=P, ranks=P, ad=P, m=5, x=P, xs=128, base=P,
             bs=96, y=P, ys=96, ws=P, wb=1 << 30)
    a.update(kw)
    d = mnb.mnb_adapter_desc(a["n"], a["k"], a["rank"], a["count"], a["dt"], a["reserved"])
    return mnb.lib.mnb_adapters_add(ctypes.byref(d), a["a"], a["b"], a["sc"], a["ranks"], a["ad"], a["m"], a["x"], a["xs"],
                                    a["base"], a["bs"], a["y"], a["ys"], a["ws"], a["wb"], None)


def verify(**kw):
    a = dict(t=P, ts=500, q=P, qs=500, ids=P, qst=P, batch=2, tokens=7, vocab=500, dt=F32, acc=P, pick=P, out=P, n=P, ws=P,
             wb=1 << 20)
    a.update(kw)
    return mnb.lib.mnb_verify_drafts(a["t"], a["ts"], a["q"], a["qs"], a["ids"], a["qst"], a["batch"], a["tokens"],
                                     a["vocab"], a["dt"], a["acc"], a["pick"], a["out"], a["n"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(dt=-1), dict(reserved=1), dict(n=-1), dict(k=0), dict(rank=0), dict(count=-1), dict(m=-1), dict(xs=127),
    dict(bs=95), dict(ys=95), dict(xs=1 << 62), dict(ys=1 << 62), dict(bs=1 << 62), dict(a=None), dict(b=None),
    dict(ad=None), dict(x=None), dict(y=None), dict(a=P + 8), dict(b=P + 8), dict(sc=P + 2), dict(ranks=P + 1),
    dict(ad=P + 2), dict(x=P + 1), dict(base=P + 1), dict(y=P + 1), dict(dt=F32, x=P + 2), dict(bs=97), dict(rank=65, ws=None),
    dict(rank=65, ws=P + 16), dict(rank=65, wb=16)])
def test_adapters_refuse(kw):
    _refused(INVALID, add, **kw)


@pytest.mark.parametrize("kw", [
    dict(rank=129), dict(n=(1 << 24) + 1, ys=1 << 25, bs=1 << 25), dict(k=(1 << 24) + 1, xs=1 << 25), dict(m=1 << 24),
    dict(m=1 << 23, n=1 << 24, ys=1 << 24, bs=1 << 24)])
def test_adapters_unsupported(kw):
    _refused(UNSUPPORTED, add, **kw)


def test_adapters_workspace():
    # few rows need none; many, or a high rank, rows of h between two launches
    few, many = mnb.mnb_adapter_desc(96, 2048, 20, 30, F16, 0), mnb.mnb_adapter_desc(96, 4096, 100, 30, F16, 0)
    assert mnb.mnb_adapters_workspace_bytes(few, 5) == 0
    if _no_device():
        _refused(DEVICE, add, m=5, k=2048, xs=2048, rank=20, count=30, ws=None, wb=0)
    for d, m, pitch in ((few, 5000, 32), (many, 1, 128), (many, 300, 128)):
        n = mnb.mnb_adapters_workspace_bytes(d, m)
        assert m * pitch * 4 <= n <= m * pitch * 4 * 8 and n % (m * pitch * 4) == 0
        kw = dict(m=m, k=d.k, xs=d.k, rank=d.rank, count=30)
        _refused(INVALID, add, wb=n - 1, **kw)
        if _no_device():
            _refused(DEVICE, add, wb=n, **kw)
    assert mnb.mnb_adapters_workspace_bytes(few, 0) == 0 and mnb.mnb_last_error() == ""
    assert mnb.mnb_adapters_workspace_bytes(few, -1) == 0 and mnb.mnb_last_error() != ""
    assert mnb.mnb_adapters_workspace_bytes(mnb.mnb_adapter_desc(96, 4096, 200, 3, F16, 0), 5) == 0


def test_nothing_to_do_is_a_noop():
    for kw in (dict(m=0, x=None), dict(n=0, ys=0, bs=0)):
        assert add(**kw) == 0 and mnb.mnb_last_variant() == "noop"
    assert verify(batch=0) == 0 and mnb.mnb_last_variant() == "noop"


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(batch=-1), dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(ts=499), dict(qs=499),
    dict(ts=1 << 61), dict(qst=None), dict(t=None), dict(ids=None), dict(acc=None), dict(pick=None), dict(out=None),
    dict(n=None), dict(t=P + 2), dict(dt=F16, t=P + 1), dict(q=P + 2), dict(ids=P + 2), dict(qst=P + 1), dict(acc=P + 2),
    dict(pick=P + 2), dict(out=P + 2), dict(n=P + 2), dict(ws=None), dict(ws=P + 16), dict(wb=31)])
def test_verify_refuses(kw):
    _refused(INVALID, verify, **kw)


def test_verify_unsupported():
    _refused(UNSUPPORTED, verify, vocab=(1 << 30) + 1, ts=1 << 31, qs=1 << 31)
    _refused(UNSUPPORTED, verify, batch=1 << 24)
    _refused(UNSUPPORTED, verify, batch=1 << 10, vocab=1 << 28, ts=1 << 28, qs=1 << 28)


def test_verify_workspace():
    for batch, vocab, chunks in ((1, 1, 1), (3, 1024, 1), (3, 1025, 2), (7, 128000, 125)):
        assert mnb.mnb_verify_workspace_bytes(batch, vocab) == 16 * batch * chunks
    assert mnb.mnb_verify_workspace_bytes(0, 5) == 0 and mnb.mnb_last_error() == ""
    assert mnb.mnb_verify_workspace_bytes(1, 0) == 0 and mnb.mnb_last_error() != ""


@pytest.mark.skipif(not _no_device(), reason="a GPU is visible")
def test_no_device_is_an_error_not_an_abort():
    for call, kw in ((add, {}), (add, dict(count=0, a=None, b=None, ws=None, wb=0)), (add, dict(sc=None, ranks=None, base=None)),
                     (verify, {}), (verify, dict(q=None)), (verify, dict(tokens=2, qst=None)),
                     (verify, dict(tokens=0, t=None, ids=None, acc=None, out=None))):
        _refused(DEVICE, call, **kw)
