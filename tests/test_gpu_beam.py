"""Selection of beam search on the GPU against the same in float64.

Bound of a score: a sum of positive terms errs by no more of itself than its terms do.  An
exponential is one of the device (2^-23 of its value), of an argument whose rounding is put back in
(what is left is below 2^-24 of a term), so the logarithm of their sum errs by 2^-22 at most; sums
and totals in 64 bits add nothing that counts, and the score is rounded once, by 2^-24 of itself.
Rows and tokens have to be equal, except that two continuations whose keys differ by less than
twice that bound may change places."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import pages_ref as R
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
LSE = 2.0 ** -22


def dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dt is None else t.to(dt)).to(DEV)


def check(logits, score, width, eos=-1, done=None, norm=None, got=None, ties=False):
    """ties: equal keys are meant, so that every index has to be equal."""
    parent, token, sc, dn = (t.cpu().numpy() for t in got)
    wp, wt, ws, wd, wk = R.beam_select(logits, score, width, eos, done, norm)
    nm = np.ones(len(wp)) if norm is None else np.asarray(norm, np.float64)
    total = R.beam_totals(logits, score, eos, done)
    for i in range(len(wp)):
        r0 = i // width * width
        if parent[i] != wp[i] or token[i] != wt[i]:
            assert not ties, (i, parent[i], token[i], wp[i], wt[i])
            key = total[parent[i], token[i]] * nm[parent[i]]
            tol = 2 * LSE * nm[r0:r0 + width].max()
            assert token[i] >= 0 and abs(key - wk[i]) <= tol, (i, key, wk[i])
            assert len({(parent[j], token[j]) for j in range(r0, r0 + width)}) == width
        if token[i] < 0:
            assert sc[i] == -np.inf and dn[i] == 0 and parent[i] == r0
            continue
        t = total[parent[i], token[i]]
        assert abs(sc[i] - t) <= LSE + 2.0 ** -24 * abs(t), (i, sc[i], t)
        assert dn[i] == int((done is not None and done[parent[i]] != 0) or token[i] == eos)
    return wp, wt


def make(rng, rows, vocab, dt, ldl=None, spread=3.0):
    x = (spread * rng.standard_normal((rows, vocab))).astype(np.float32)
    x = x.astype(np.float16 if dt == "f16" else np.float32)
    wide = np.full((rows, ldl or vocab), np.nan, x.dtype)
    wide[:, :vocab] = x
    return x, dev(wide)[:, :vocab]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("req,width,vocab,ldl", [
    (1, 1, 1, 1), (1, 1, 7, 9), (2, 32, 1, 4), (1, 32, 20, 21), (3, 4, 2049, 2051), (1, 4, 32000, 32000),
    (5, 5, 8191, 8193), (2, 8, 8193, 8200), (40, 2, 4097, 4099), (7, 32, 10007, 10007),
    (64, 4, 1000, 1024), (1, 16, 131072, 131075), (9, 32, 32768, 32768)])
def test_random(req, width, vocab, ldl, dt):
    rng = np.random.default_rng(req * 1000 + vocab)
    rows = req * width
    x, logits = make(rng, rows, vocab, dt, ldl)
    score = -20 * rng.random(rows).astype(np.float32)
    eos = int(rng.integers(0, vocab))
    done = (rng.random(rows) < 0.2).astype(np.int32)
    norm = (0.2 + rng.random(rows)).astype(np.float32)
    ws = B.beam_workspace(req, width, vocab, DEV)
    for d, nm in ((None, None), (done, None), (None, norm), (done, norm)):
        say(f"case: beams req={req} width={width} vocab={vocab} {dt} done={d is not None} "
            f"norm={nm is not None}")
        got = B.beam_select(logits, dev(score), width, eos, None if d is None else dev(d),
                            None if nm is None else dev(nm), ws=ws)
        check(x, score, width, eos, d, nm, got)
        assert not ws[:65536].any()


@pytest.mark.parametrize("width", [1, 3, 8, 32])
def test_ties(width):
    """Equal logits by the thousand, equal rows, rows of one value: the lowest indices."""
    rng = np.random.default_rng(width)
    vocab = 20011
    rows = []
    rows.append(np.zeros(vocab))                                  # every total equal
    rows.append(rng.integers(0, 3, vocab))                        # a third of them
    rows.append(np.where(np.arange(vocab) % 4096 == 4095, 1, 0))  # a few, far apart
    last = np.zeros(vocab)
    last[-width:] = 2
    rows.append(last)
    for x in rows:
        x = np.repeat(x[None].astype(np.float16), 2 * width, 0)   # equal rows, at every alignment
        wide = np.zeros((2 * width, vocab + 2), np.float16)
        wide[:, :vocab] = x
        score = np.zeros(2 * width, np.float32)
        say(f"case: ties width={width}")
        got = B.beam_select(dev(wide)[:, :vocab], dev(score), width)
        check(x, score, width, got=got, ties=True)


def test_first_step_and_dead_rows():
    """-inf scores, NaN scores, norms that are none: such rows have no continuation."""
    rng = np.random.default_rng(5)
    width, vocab = 6, 5000
    x, logits = make(rng, 4 * width, vocab, "f32")
    score = np.full(4 * width, -np.inf, np.float32)
    score[0] = score[width + 2] = 0.0
    score[2 * width + 1] = np.nan                                 # request 2 has nothing at all
    score[3 * width:] = -1.0
    norm = np.ones(4 * width, np.float32)
    norm[3 * width:3 * width + 3] = 0.0, -1.0, np.inf
    norm[3 * width + 3] = np.nan
    got = B.beam_select(logits, dev(score), width, norm=dev(norm))
    wp, wt = check(x, score, width, norm=norm, got=got)
    assert (wt[2 * width:3 * width] == -1).all() and (wp[2 * width:3 * width] == 2 * width).all()
    # fewer continuations than beams
    x, logits = make(rng, 8, 3, "f16")
    score = np.array([0] + [-np.inf] * 7, np.float32)
    got = B.beam_select(logits, dev(score), 8)
    wp, wt = check(x, score, 8, got=got)
    assert (wt >= 0).sum() == 3
    # every beam is done
    done = np.ones(8, np.int32)
    score = -np.arange(8, dtype=np.float32)[::-1].copy()
    got = B.beam_select(logits, dev(score), 8, eos=1, done=dev(done))
    wp, _ = check(x, score, 8, 1, done, got=got)
    assert wp.tolist() == list(range(7, -1, -1))


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_masked_and_infinite_logits(dt):
    rng = np.random.default_rng(11)
    width, vocab = 4, 9001
    x, _ = make(rng, 5 * width, vocab, dt)
    x[:width, 50:] = -np.inf                   # most of the vocabulary banned
    x[width:2 * width, 1:] = -np.inf           # one token is left
    x[2 * width:3 * width] = -np.inf           # none
    x[3 * width, 4000] = np.inf
    x[3 * width + 1, 100:200] = np.nan
    x[3 * width + 2, :] = np.finfo(x.dtype).min
    x[4 * width:, ::2] = np.finfo(x.dtype).min  # masks of the type's lowest value
    score = -rng.random(5 * width).astype(np.float32)
    got = B.beam_select(dev(x), dev(score), width)
    wp, wt = check(x, score, width, got=got)
    assert (wt[2 * width:3 * width] == -1).all()


@pytest.mark.parametrize("order", ["up", "down", "saw", "peak", "steps"])
@pytest.mark.parametrize("width,vocab", [(2, 40000), (32, 140000)])
def test_logits_in_order(order, width, vocab):
    """Every element above all before it, the best ones all in one piece, pieces of equal values:
    lists that fill, whose bounds have to rise."""
    rng = np.random.default_rng(width)
    at = np.arange(vocab, dtype=np.float64)
    x = {"up": at / vocab * 20, "down": -at / vocab * 20, "saw": at % 4099 / 200,
         "peak": -np.abs(at - vocab / 3) / 500, "steps": at // 700 / 10}[order]
    rows = 3 * width
    x = np.repeat(x[None], rows, 0).astype(np.float32)
    x[2 * width:] += 0.01 * rng.standard_normal((width, vocab)).astype(np.float32)
    score = np.zeros(rows, np.float32)
    score[width:] = -rng.random(2 * width).astype(np.float32)
    for dt in (np.float32, np.float16):
        say(f"case: logits in order, {order} width={width} {dt.__name__}")
        got = B.beam_select(dev(x.astype(dt)), dev(score), width)
        check(x.astype(dt), score, width, got=got)


def test_rows_past_32_bits():
    say("case: beams over rows of 2.4 GB")
    rng = np.random.default_rng(8)
    wide = torch.empty((4, 600_000_000), dtype=torch.float32, device=DEV)
    x = (3 * rng.standard_normal((4, 5000))).astype(np.float32)
    wide[:, :5000] = dev(x)
    score = -rng.random(4).astype(np.float32)
    got = B.beam_select(wide[:, :5000], dev(score), 4)
    check(x, score, 4, got=got)


def test_close_totals_of_different_rows():
    """Rows whose best totals differ by 2^-18 (sixteen times what a sum may err by), the
    probabilities spread over the whole vocabulary."""
    rng = np.random.default_rng(13)
    width, vocab = 8, 60000
    x = rng.standard_normal((width, vocab)).astype(np.float32)
    x[:, 777] = 9.0
    t = R.beam_totals(x, np.zeros(width), -1)[:, 777]
    order = rng.permutation(width)
    score = (-5.0 - t - order * 2.0 ** -18).astype(np.float32)
    # what rounding the scores to fp32 leaves of the distances
    now = np.sort((t + score)[np.argsort(order)])
    assert np.diff(now).min() > 2.0 ** -19
    got = B.beam_select(dev(x), dev(score), width)
    wp, wt = check(x, score, width, got=got, ties=True)
    assert (wt == 777).all() and np.array_equal(wp, np.argsort(order))


def test_calls_share_a_workspace_in_any_order():
    rng = np.random.default_rng(17)
    ws = B.beam_workspace(40, 8, 20000, DEV)
    ws[65536:] = 0xFF
    for req, width, vocab, dt in ((40, 8, 20000, "f32"), (1, 8, 20000, "f16"), (3, 2, 777, "f32"),
                                  (40, 1, 20000, "f16"), (39, 8, 19999, "f16"), (1, 1, 1, "f32"),
                                  (20, 8, 20000, "f32")):
        x, logits = make(rng, req * width, vocab, dt)
        score = -rng.random(req * width).astype(np.float32)
        say(f"case: one workspace req={req} width={width} vocab={vocab} {dt}")
        got = B.beam_select(logits, dev(score), width, ws=ws)
        check(x, score, width, got=got)
        assert not ws[:65536].any()
