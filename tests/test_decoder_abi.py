"""Argument checks of the norm, the 4-bit cache and the attention through the C
ABI.  No GPU: every check runs on the host before any HIP call, and a
well-formed request without a device returns MNB_ERR_DEVICE."""
import ctypes

import pytest

from block_wise_int4_amd import mnb

INVALID, UNSUPPORTED, DEVICE = mnb.MNB_ERR_INVALID_ARGUMENT, mnb.MNB_ERR_UNSUPPORTED, mnb.MNB_ERR_DEVICE
P = 1 << 20     # an aligned address that nothing reads
F16, F32 = mnb.MNB_F16, mnb.MNB_F32


def desc(**kw):
    d = dict(q_heads=8, kv_heads=2, head_dim=128, group_size=64, page_size=64, num_pages=10)
    d.update(kw)
    return mnb.kv4_desc(*(d[k] for k in ("q_heads", "kv_heads", "head_dim", "group_size", "page_size", "num_pages")))


def norm(**kw):
    a = dict(x=P, xs=256, r=P, rs=256, w=P, m=4, k=256, dt=F16, eps=1e-5, kind=0, out=P, sc=None, ro=P)
    a.update(kw)
    return mnb.lib.mnb_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["m"], a["k"], a["dt"], a["eps"], a["kind"],
                                a["out"], a["sc"], a["ro"], None)


def append(d=None, **kw):
    a = dict(cache=P, table=P, ts=4, kl=P, qs=P, batch=2, tokens=5, dt=F16, q=P, q_s=1024, k=P, k_s=256, v=P, v_s=256,
             cos=P, sin=P, rows=100, rot=64, inter=0, qo=P)
    a.update(kw)
    d = d or desc()
    return mnb.lib.mnb_kv4_append(ctypes.byref(d), a["cache"], a["table"], a["ts"], a["kl"], a["qs"], a["batch"],
                                  a["tokens"], a["dt"], a["q"], a["q_s"], a["k"], a["k_s"], a["v"], a["v_s"], a["cos"],
                                  a["sin"], a["rows"], a["rot"], a["inter"], a["qo"], None)


def read(d=None, **kw):
    a = dict(cache=P, table=P, ts=4, kl=P, qs=P, batch=2, tokens=5, dt=F16, k=P, v=P)
    a.update(kw)
    d = d or desc()
    return mnb.lib.mnb_kv4_read(ctypes.byref(d), a["cache"], a["table"], a["ts"], a["kl"], a["qs"], a["batch"],
                                a["tokens"], a["dt"], a["k"], a["v"], None)


def attend(d=None, **kw):
    a = dict(cache=P, table=P, ts=4, kl=P, qs=P, batch=2, tokens=5, mq=3, mk=250, dt=F16, q=P, q_s=1024, scale=0.1,
             causal=1, window=0, out=P, lse=None, ws=P, wb=1 << 30)
    a.update(kw)
    d = d or desc()
    return mnb.lib.mnb_attention_kv4(ctypes.byref(d), a["cache"], a["table"], a["ts"], a["kl"], a["qs"], a["batch"],
                                     a["tokens"], a["mq"], a["mk"], a["dt"], a["q"], a["q_s"], a["scale"], a["causal"],
                                     a["window"], a["out"], a["lse"], a["ws"], a["wb"], None)


def _no_device():
    try:
        import torch
        return not torch.cuda.is_available()
    except Exception:
        return True


def _refused(status, call, **kw):
    assert call(**kw) == status, (call.__name__, kw, mnb.mnb_last_error())
    assert mnb.mnb_last_error().startswith("mnb: "), kw


@pytest.mark.parametrize("kw", [
    dict(dt=7), dict(kind=3), dict(kind=-1), dict(m=-1), dict(k=0), dict(k=1 << 31), dict(m=1 << 31), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(sc=P), dict(kind=1), dict(kind=2), dict(xs=255), dict(rs=255),
    dict(xs=1 << 62), dict(x=None), dict(w=None), dict(out=None), dict(x=P + 1), dict(r=P + 1), dict(ro=P + 1),
    dict(w=P + 1), dict(out=P + 1), dict(kind=1, sc=P + 2), dict(dt=F32, x=P + 2), dict(kind=1, sc=P, out=P + 1)])
def test_norm_refuses(kw):
    _refused(INVALID, norm, **kw)


def test_norm_without_rows_is_a_noop():
    assert norm(m=0) == 0 and mnb.mnb_last_variant() == "noop"


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(q_heads=7), INVALID), (dict(num_pages=-1), INVALID),
    (dict(num_pages=1 << 31), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(group_size=16), UNSUPPORTED), (dict(head_dim=64, group_size=128), UNSUPPORTED),
    (dict(page_size=16), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(q_heads=1 << 17), UNSUPPORTED)])
def test_every_call_refuses_a_bad_descriptor(kw, status):
    for call in (append, read, attend):
        _refused(status, call, d=desc(**kw))
    with pytest.raises(mnb.MnbError):
        mnb.mnb_kv4_cache_bytes(desc(**kw))
    assert mnb.mnb_attention_kv4_workspace_bytes(desc(**kw), 1, 1, 1, 100) == 0
    assert mnb.mnb_last_error() != ""


def test_cache_size_is_the_documented_one():
    for D, g, page in ((64, 32, 32), (128, 128, 64), (128, 64, 256), (256, 32, 128)):
        d = desc(head_dim=D, group_size=g, page_size=page, num_pages=7, kv_heads=4, q_heads=8)
        assert mnb.mnb_kv4_cache_bytes(d) == 7 * 4 * (page // 32) * (32 * D + 256 * (D // g))
    big = desc(num_pages=(1 << 31) - 1)
    assert mnb.mnb_kv4_cache_bytes(big) > 1 << 40
    with pytest.raises(mnb.MnbError):
        mnb.mnb_kv4_cache_bytes(desc(num_pages=0))


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(batch=-1), dict(tokens=-1), dict(batch=1 << 31), dict(cos=None), dict(sin=None), dict(inter=2),
    dict(rot=0), dict(rot=144), dict(rows=0), dict(q=None), dict(qo=None), dict(k_s=255), dict(v_s=255), dict(q_s=1023),
    dict(table=None), dict(kl=None), dict(qs=None), dict(ts=0), dict(k=None), dict(v=None), dict(cache=None),
    dict(cache=P + 16), dict(k=P + 1), dict(table=P + 2), dict(qs=P + 1), dict(cos=P + 1), dict(dt=F32, v=P + 2),
    dict(tokens=1 << 40)])
def test_append_refuses(kw):
    _refused(INVALID, append, **kw)


def test_append_unsupported():
    _refused(UNSUPPORTED, append, rot=24)
    _refused(UNSUPPORTED, append, tokens=(1 << 31) - 1, k_s=256, q_s=1024)


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(batch=-1), dict(tokens=-1), dict(table=None), dict(kl=None), dict(qs=None), dict(ts=0),
    dict(cache=None), dict(cache=P + 128), dict(k=P + 1), dict(dt=F32, v=P + 2)])
def test_read_refuses(kw):
    _refused(INVALID, read, **kw)


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(batch=-1), dict(tokens=-1), dict(mq=-1), dict(mk=-1), dict(causal=2), dict(window=-1),
    dict(window=5, causal=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_s=1023), dict(table=None),
    dict(kl=None), dict(qs=None), dict(ts=0), dict(q=None), dict(out=None), dict(cache=None), dict(cache=P + 16),
    dict(lse=P + 2), dict(out=P + 1), dict(ws=None), dict(ws=P + 16), dict(wb=16)])
def test_attention_refuses(kw):
    # many keys and few rows: a call that needs its workspace
    _refused(INVALID, attend, mk=kw.pop("mk", 100000), **kw)


def test_attention_unsupported():
    _refused(UNSUPPORTED, attend, batch=70000, tokens=70000)
    _refused(UNSUPPORTED, attend, mk=(1 << 30) + 1)
    _refused(UNSUPPORTED, attend, mq=1 << 30)


def test_empty_requests_are_noops():
    for kw in (dict(tokens=0), dict(batch=0)):
        for call in (append, read, attend):
            assert call(**kw) == 0 and mnb.mnb_last_variant() == "noop"
    assert attend(mq=0) == 0 and read(k=None, v=None) == 0


def test_workspace_is_bounded_and_enough():
    d = desc()
    n = mnb.mnb_attention_kv4_workspace_bytes(d, 1, 1, 1, 100000)
    assert 0 < n < 1 << 28
    if _no_device():
        assert attend(batch=1, tokens=1, mq=1, mk=100000, wb=n) == DEVICE
    _refused(INVALID, attend, batch=1, tokens=1, mq=1, mk=100000, wb=n - 1)
    assert mnb.mnb_attention_kv4_workspace_bytes(d, 0, 0, 0, 0) == 0


def test_codes_product_refuses():
    w = mnb.desc(64, 256, 32, True, F16)

    def call(w=w, rep=P, codes=P, sc=P, m=4, bias=None, y=P):
        return mnb.lib.mnb_gemm_accuracy4_codes(ctypes.byref(w), rep, codes, sc, m, bias, y, None)

    for kw in (dict(m=-1), dict(m=1 << 31), dict(rep=None), dict(rep=P + 16), dict(codes=None), dict(codes=P + 2),
               dict(sc=None), dict(sc=P + 2), dict(y=None), dict(y=P + 2), dict(bias=P + 2)):
        _refused(INVALID, call, **kw)
    _refused(UNSUPPORTED, call, w=mnb.desc(64, 250, 32, True, F16))
    assert call(m=0) == 0


@pytest.mark.skipif(not _no_device(), reason="a GPU is visible")
def test_no_device_is_an_error_not_an_abort():
    for call in (norm, append, read, attend):
        _refused(DEVICE, call)
