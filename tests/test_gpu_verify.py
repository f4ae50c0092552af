"""Verification of drafted tokens on the GPU: every token equal to the 64-bit oracle's."""
import numpy as np
import pytest

from oracle import requests as o
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def softmax(x):
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def inputs(rng, counts, vocab, dt, before=0, behind=0, close=0.6):
    """Target and draft distributions, drafts from the draft's, random numbers; rows of no sequence on both sides."""
    kind = np.float16 if dt == "f16" else np.float32
    tokens = before + sum(counts) + behind
    logits = 2.5 * rng.normal(size=(tokens, vocab))
    target, draft = softmax(logits).astype(kind), softmax(logits + close * rng.normal(size=logits.shape)).astype(kind)
    ids = rng.integers(0, vocab, tokens).astype(np.int32)
    for i in range(1, tokens):
        w = draft[i - 1].astype(np.float64)
        ids[i] = rng.choice(vocab, p=w / w.sum()) if w.sum() > 0 else 0
    q_start = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    return target, draft, ids, q_start, rng.random(tokens).astype(np.float32), rng.random(len(counts)).astype(np.float32)


def run(mnb, target, draft, ids, q_start, accept, pick, stream=None):
    t = G.torch()
    out = t.full((len(ids),), 77, dtype=t.int32, device="cuda")
    accepted = t.full((len(pick),), 77, dtype=t.int32, device="cuda")
    size = mnb.mnb_verify_workspace_bytes(len(pick), target.shape[1])
    ws = t.full((size,), 0xFF, dtype=t.uint8, device="cuda")
    up = [None if v is None else G.to_dev(v) if isinstance(v, np.ndarray) else v for v in (target, draft, ids, q_start, accept, pick)]
    mnb.mnb_verify_drafts(up[0], up[2], up[4], up[5], out, accepted, q_start=up[3], draft=up[1], workspace=ws, stream=stream)
    return out, accepted


def check(mnb, target, draft, ids, q_start, accept, pick):
    out, accepted = run(mnb, target, draft, ids, q_start, accept, pick)
    want, counts = o.verify(target, draft, ids, q_start, accept, pick, np.full(len(ids), 77, np.int32))
    assert accepted.cpu().numpy().tolist() == counts.tolist()
    assert out.cpu().numpy().tolist() == want.tolist()
    return counts


CASES = [  # rows of the sequences, vocabulary
    ([1], 1), ([2], 2), ([3, 1], 5), ([1, 5, 0, 2], 100), ([4], 4095), ([4, 4], 4096), ([9, 1, 3], 4097), ([6] * 20, 1000),
    ([3, 2], 1023), ([3, 2], 1025), ([2], 65537),
    ([5, 0, 0, 7], 50257), ([70, 130], 33), ([3], 200001), ([0, 0], 10), ([2] * 300, 40),
    ([1, 4, 2], 16385), ([3], 32769), ([1] * 255 + [0, 2, 3], 33000),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("case", CASES, ids=["%d-%d-%d" % (len(c[0]), c[0][0], c[1]) for c in CASES])
def test_against_the_oracle(mnb, case, certain, dt):
    counts, vocab = case
    rng = np.random.default_rng((980, len(counts), counts[0], vocab))
    target, draft, *rest = inputs(rng, counts, vocab, dt, before=2, behind=3)
    check(mnb, target, None if certain else draft, *rest)


@pytest.mark.parametrize("certain", [False, True])
def test_long_runs_of_accepted_drafts(mnb, certain):
    """Refusals at every place, the borders of 64 drafts among them, and none."""
    rng = np.random.default_rng(981)
    target, draft, ids, q_start, accept, pick = inputs(rng, [140] * 12, 17, "f32")
    accept[:] = 0
    for b, stop in enumerate([0, 1, 62, 63, 64, 65, 127, 128, 129, 138, None, None]):
        if stop is not None:
            accept[140 * b + stop] = 1e9
    counts = check(mnb, target, None if certain else draft, ids, q_start, accept, pick)
    assert counts.tolist() == [0, 1, 62, 63, 64, 65, 127, 128, 129, 138, 139, 139]


def test_one_row_each_without_offsets(mnb):
    rng = np.random.default_rng(982)
    target, _, ids, _, accept, pick = inputs(rng, [1] * 50, 5000, "f32")
    check(mnb, target, None, ids, None, accept, pick)


def test_draws_on_exact_borders(mnb):
    """Weights that are multiples of 2^-10 and picks on their sums: the next token, never the one that ends there."""
    rng = np.random.default_rng(983)
    vocab = 9000
    w = np.zeros(vocab, np.float32)
    at = np.sort(rng.choice(vocab, 256, replace=False))
    at[100:103] = [4095, 4096, 4097] if not set([4095, 4096, 4097]) & set(at) else at[100:103]
    at = np.unique(at)
    w[at] = 2.0 ** -10 * rng.integers(1, 5, len(at))
    w[at[-1]] += np.float32(1.0 - w.sum())
    assert w.sum(dtype=np.float64) == 1.0
    sums = np.cumsum(w.astype(np.float64))[at]
    pick = np.concatenate([[0.0], sums[:-1], sums[:-1] - 2.0 ** -12]).astype(np.float32)
    B = len(pick)
    check(mnb, np.tile(w, (B, 1)), None, np.zeros(B, np.int32), None, np.zeros(B, np.float32), pick)


def test_picks_outside_their_range(mnb):
    rng = np.random.default_rng(984)
    pick = np.array([0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, np.inf, -1.0, -np.inf, np.nan, -0.0], np.float32)
    w = softmax(rng.normal(size=(9, 6000))).astype(np.float32)
    w[:, 5990:] = 0
    w[:, :3] = 0
    check(mnb, w, None, np.zeros(9, np.int32), None, np.zeros(9, np.float32), pick)


def test_nothing_left_and_bad_probabilities(mnb):
    """A refused draft of equal distributions draws from p; NaN, infinite and negative values count as 0; rows without
    a weight draw -1; drafts outside the vocabulary are refused."""
    rng = np.random.default_rng(985)
    vocab, counts = 300, [3] * 8
    target, draft, ids, q_start, accept, pick = inputs(rng, counts, vocab, "f32")
    accept[:] = 0.5
    draft[0:3] = target[0:3]
    accept[0] = 1.0                                     # u q < p does not hold where q = p
    target[3:6, 10:60], draft[3:6, 100:110] = np.nan, np.nan
    target[6:9, 10:60], draft[6:9, 100:110] = np.inf, -np.inf
    target[9:12, 10:60], draft[9:12, 100:110] = -1.0, -0.5
    target[12:15] = 0
    target[15:18] = np.nan
    ids[19] = -3
    ids[22], ids[23] = vocab, 1 << 30
    for certain in (False, True):
        check(mnb, target, None if certain else draft, ids, q_start, accept, pick)
    accept[:] = np.nan
    assert (check(mnb, target, draft, ids, q_start, accept, pick) == 0).all()


def test_offsets_out_of_range_stay_inside(mnb):
    rng = np.random.default_rng(986)
    target, draft, ids, _, accept, pick = inputs(rng, [4] * 4, 50, "f32")
    for q_start in ([-5, 3, 2, 9, 40], [0, 16, 16, 1 << 30, 5], [12, 30, -1, 0, 2]):
        check(mnb, target, draft, ids, np.array(q_start, np.int32), accept, pick)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_rows_of_wider_arrays(mnb, dt):
    t = G.torch()
    rng = np.random.default_rng(987)
    target, draft, *rest = inputs(rng, [5, 3], 4500, dt)
    want = run(mnb, target, draft, *rest)
    wide = t.full((8, 9100), float("nan"), dtype=t.float16 if dt == "f16" else t.float32, device="cuda")
    wide[:, 1:4501], wide[:, 4503:9003] = G.to_dev(target), G.to_dev(draft)
    got = run(mnb, wide[:, 1:4501], wide[:, 4503:9003], *rest)
    assert t.equal(want[0], got[0]) and t.equal(want[1], got[1])


def test_replays_and_streams_give_the_eager_tokens(mnb):
    t = G.torch()
    rng = np.random.default_rng(988)
    target, draft, ids, q_start, accept, pick = (G.to_dev(v) for v in inputs(rng, [5, 1, 8], 30000, "f32"))
    out, accepted = t.empty_like(ids), t.empty(3, dtype=t.int32, device="cuda")
    ws = t.empty(mnb.mnb_verify_workspace_bytes(3, 30000), dtype=t.uint8, device="cuda")

    def issue(stream):
        mnb.mnb_verify_drafts(target, ids, accept, pick, out, accepted, q_start=q_start, draft=draft, workspace=ws,
                              stream=stream)

    issue(t.cuda.current_stream())
    t.cuda.synchronize()
    eager = out.clone(), accepted.clone()
    s = t.cuda.Stream()
    out.fill_(99)
    s.wait_stream(t.cuda.current_stream())
    issue(s)
    s.synchronize()
    assert t.equal(out, eager[0]) and t.equal(accepted, eager[1])
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            issue(s)
    t.cuda.current_stream().wait_stream(s)
    for i in range(3):
        accept.copy_(t.rand_like(accept))               # new numbers in the same buffers
        pick.copy_(t.rand_like(pick))
        issue(t.cuda.current_stream())
        t.cuda.synchronize()
        want = out.clone(), accepted.clone()
        out.fill_(99)
        accepted.fill_(99)
        ws.fill_(0xFF)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(out, want[0]) and t.equal(accepted, want[1])


def test_binding_refuses_wrong_tensors(mnb):
    t = G.torch()
    i, f = dict(dtype=t.int32, device="cuda"), dict(device="cuda")
    good = dict(target=t.rand(4, 60, **f), ids=t.zeros(4, **i), accept=t.zeros(4, **f), pick=t.zeros(2, **f),
                out=t.zeros(4, **i), accepted=t.zeros(2, **i), q_start=t.tensor([0, 2, 4], **i), draft=t.rand(4, 60, **f),
                workspace=t.zeros(4096, dtype=t.uint8, device="cuda"))
    mnb.mnb_verify_drafts(**good)
    for name, bad in (("target", good["target"].double()), ("target", good["target"].t()), ("draft", good["draft"][:3]),
                      ("draft", good["draft"].half()), ("ids", good["ids"].long()), ("ids", good["ids"][:3]),
                      ("accept", good["accept"].half()), ("accept", good["accept"][:2]), ("pick", good["pick"].double()),
                      ("pick", good["pick"][:1]), ("out", good["out"][:3]), ("accepted", good["accepted"][:1]),
                      ("q_start", good["q_start"].long()), ("q_start", good["q_start"][:2]), ("ids", good["ids"].cpu())):
        with pytest.raises(ValueError):
            mnb.mnb_verify_drafts(**dict(good, **{name: bad}))
    for bad in (dict(workspace=None), dict(q_start=None)):
        with pytest.raises(mnb.MnbError):
            mnb.mnb_verify_drafts(**dict(good, **bad))


@pytest.mark.parametrize("vocab, batch", [(3, (1 << 22) + 5), (2049, 70000), (15400, 1500)])
def test_many_sequences(mnb, vocab, batch):
    """Sequences of one row: the token alone.  Weights are whole numbers, so every sum is exact in any order."""
    t = G.torch()
    gen = t.Generator(device="cuda").manual_seed(986)
    p = t.empty(batch, vocab, dtype=t.float16, device="cuda").random_(0, 4, generator=gen)
    pick = t.rand(batch, device="cuda", generator=gen)
    ids = t.zeros(batch, dtype=t.int32, device="cuda")
    out, accepted = run(mnb, p, None, ids, None, t.zeros(batch, device="cuda"), pick)
    assert not accepted.any()
    for i in range(0, batch, 1 << 17):
        upto = p[i:i + (1 << 17)].to(t.float32).cumsum(1)
        over = upto.double() > (pick[i:i + (1 << 17)].double() * upto[:, -1].double())[:, None]
        want = t.where(over.any(1), over.to(t.uint8).argmax(1).to(t.int32), t.tensor(-1, dtype=t.int32, device="cuda"))
        assert t.equal(out[i:i + (1 << 17)], want)
