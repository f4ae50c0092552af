"""Every form of the attention's kernels: each head_dim, groups and type, with as many rows a key head and sequences as
take each of its row layouts."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_kv4 import dev, desc_of, sequences
from tests.test_gpu_kv4_attention import check, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


HEADS = [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 64), (256, 32)]   # head_dim, group
FORMS = {  # q heads, kv heads, new tokens, cached with them, bound of the keys, variant
    "4 rows": (8, 2, [1, 1], [200, 33], 200, "attention_kv4"),
    "8 rows": (4, 1, [2, 1], [199, 31], 199, "attention_kv4"),
    "16 rows": (6, 2, [5, 3, 1], [160, 64, 1], 160, "attention_kv4"),
    "32 rows": (8, 2, [8, 5], [330, 70], 2000, "attention_kv4_split"),
    "4 rows, split": (2, 1, [2, 2], [420, 256], 2000, "attention_kv4_split"),
    "8 rows, split": (4, 2, [4, 3], [300, 513], 2000, "attention_kv4_split"),
    "16 rows, split": (3, 1, [5, 2], [290, 600], 2000, "attention_kv4_split"),
    "many rows": (2, 1, [150, 17, 1], [200, 60, 33], 200, "attention_kv4_prompt"),
    "many rows, split": (2, 1, [70, 3], [640, 300], 1500, "attention_kv4_prompt_split"),
    # two row tiles by two heads by 64 sequences: a workgroup for every CU with two column tiles a wave
    "many rows, whole chip": (4, 2, [150] + [1, 2, 3] * 21, [200] + [3, 40, 5] * 21, 200, "attention_kv4_prompt"),
}


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_").replace(",", "") for f in FORMS])
@pytest.mark.parametrize("D,group", HEADS)
def test_every_form(mnb, D, group, form, dt):
    H, Hkv, new, lens, max_kv, variant = FORMS[form]
    rng = np.random.default_rng((960, D, group, sum(new)))
    table, pages = sequences(rng, lens, 64)
    geo = o.Geometry(H, Hkv, D, group, 64, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (1.5 * rng.normal(size=(q_start[-1], H, D))).astype(np.float16 if dt == "f16" else np.float32)
    for window in (0, 45):
        check(mnb, geo, cache, vmax, table, lens, q_start, q, D ** -0.5, window=window, max_kv=max_kv)
    took = mnb.mnb_last_variant()
    if D == 256 or D // group > 2:     # up to 16 rows always by the few-row kernels' splits, more by the many-row kernel
        assert took.startswith("attention_kv4_prompt" if "32" in form or "many" in form else "attention_kv4")
    else:
        assert took == variant


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_many_rows_over_long_keys(mnb, dt):
    """Two column tiles a wave through many stages, pages of several sizes, a prefix and its tail in one block."""
    rng = np.random.default_rng(961)
    for page, group in ((32, 128), (256, 64)):
        new, lens = [130] + [1] * 63, [1100] + [7] * 63
        table, pages = sequences(rng, lens, page)
        geo = o.Geometry(4, 2, 128, group, page, pages)
        cache, vmax = make_cache(rng, geo, table, lens)
        q_start = np.concatenate([[0], np.cumsum(new)])
        q = (1.5 * rng.normal(size=(q_start[-1], 4, 128))).astype(np.float16 if dt == "f16" else np.float32)
        check(mnb, geo, cache, vmax, table, lens, q_start, q, 128 ** -0.5)
        assert mnb.mnb_last_variant() == "attention_kv4_prompt"


def guarded(t, n, dtype, fill):
    """n elements 256-byte aligned between two guards of 4096, and a check that those are untouched."""
    buf = t.full((n + 8192,), fill, dtype=dtype, device="cuda")
    return buf[4096:4096 + n], lambda: bool((buf[:4096] == fill).all() and (buf[4096 + n:] == fill).all())


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("max_kv", [150, 5000])
@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("bad", ["length past the table", "length past the bound", "negative length", "pages outside the cache",
                                 "offset past the rows"])
def test_a_malformed_sequence_harms_only_itself(mnb, bad, new, max_kv, dt):
    """The sequences beside it are as they should be, and nothing is written outside the outputs, the rows that belong to
    sequences and a workspace of exactly the size asked for."""
    t = G.torch()
    rng = np.random.default_rng(962)
    lens, D, H = [150, 90, 120], 128, 4
    table, pages = sequences(rng, lens, 32)
    geo = o.Geometry(H, 2, D, 64, 32, pages)
    cache, vmax = make_cache(rng, geo, table, lens)
    T = 3 * new + 3                                   # three rows of no sequence
    q_start = np.array([1, 1 + new, 1 + 2 * new, 1 + 3 * new])
    q = (1.5 * rng.normal(size=(T, H, D))).astype(np.float16 if dt == "f16" else np.float32)
    w, wl, size, reach = o.attention(geo, cache, table, lens, q_start, q, 0.1)
    tol = o.attention_tolerance(size, reach, 150, D, dt == "f16", vmax)
    hurt = 1
    kv, start, tab = np.array(lens, np.int32), q_start.astype(np.int32), table.copy()
    if bad == "length past the table":
        kv[1] = 32 * table.shape[1] + 1
    elif bad == "length past the bound":
        kv[1] = 1 << 30
    elif bad == "negative length":
        kv[1] = -5
    elif bad == "pages outside the cache":
        tab[1, :3] = [1 << 30, -7, pages]
    else:
        hurt, start[3] = 2, 1 << 30
    d = desc_of(mnb, geo)
    n = mnb.mnb_attention_kv4_workspace_bytes(d, 3, T, new, max_kv)
    ws, ws_kept = guarded(t, n, t.uint8, 0xA5)
    dq = dev(q)
    out, out_kept = guarded(t, T * H * D, dq.dtype, 7.0)
    lse, lse_kept = guarded(t, T * H, t.float32, 7.0)
    mnb.mnb_attention_kv4(d, dev(cache), dq, dev(tab), dev(kv), dev(start), new, max_kv, out.view(T, H, D), 0.1,
                          lse=lse.view(T, H), workspace=ws, workspace_bytes=n)
    t.cuda.synchronize()
    assert out_kept() and lse_kept() and ws_kept()
    got, gl = G.host(out.view(T, H, D)), G.host(lse.view(T, H))
    rows = np.concatenate([np.arange(q_start[b], q_start[b + 1]) for b in range(3) if b != hurt])
    assert (np.abs(got[rows] - w[rows]) <= tol[rows]).all()
    assert (np.abs(gl[rows] - wl[rows]) <= o.lse_tolerance(wl[rows], reach[rows], 150, D)).all()
    none = [0] + list(range(q_start[3], T) if hurt == 1 else [])
    assert (got[none] == 7.0).all() and (gl[none] == 7.0).all()
