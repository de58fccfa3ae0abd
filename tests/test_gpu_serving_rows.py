"""A row of the attention depends on nothing but the keys that it sees: pages of much larger value
scales, NaN codes and NaN scales that other rows of the same wave see must not change it.

Bound of a row, in its own terms (a_j = w_j vscale_j, the size of key j's contribution): each score
errs as its fp32 sum does, which its weight follows; the exponent's argument and value add
2^-22 (2 + |s_j| + |s_max|); two f16 values hold a weight to 2^-21 of itself or 2^-37 of the row's
largest contribution; sums err as in serving_ref."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import serving_ref as R
from tests.gpu_helpers import DEV, say
from tests.test_gpu_serving import KINDS, OUT, Cache, ints

pytestmark = pytest.mark.gpu
EPS = R.EPS


def row_reference(c, Q, new, lengths, group, window, sinks, out):
    """(O, bound) of (n_tok, q_heads, dim); NaN codes and scales of keys that a row sees make it
    NaN there."""
    dim, P, H = c.dim, c.page, c.heads * group
    Q = Q.reshape(-1, H, dim)
    o, bound = np.zeros(Q.shape), np.zeros(Q.shape)
    t = 0
    for r, n in enumerate(new):
        j = np.arange(lengths[r])
        pg = c.table[r, j // P]
        for i in range(n):
            p = lengths[r] - n + i
            seen = (j <= p) & ((p - j < window) | (j < sinks) if window > 0 else True)
            for h in range(c.heads):
                kk = R.decode(c.k[pg, h, j % P], c.kind)[seen] * c.ks[pg, h, None][seen].astype(float)
                cc = R.decode(c.v[pg, h, :, j % P], c.kind)[seen]
                ss = c.vs[pg, h][seen].astype(np.float64)
                for x in range(h * group, (h + 1) * group):
                    s = kk @ Q[t, x] * dim ** -0.5
                    es = (8 * np.sqrt(dim) + 8) * EPS * (np.abs(kk) @ np.abs(Q[t, x])) * dim ** -0.5
                    w = np.exp(s - s.max())
                    a, l = w * ss, w.sum()
                    rel = es + es.max() + 2.0 ** -22 * (2 + np.abs(s) + abs(s.max())) + 2.0 ** -21
                    ea = a * rel + 2.0 ** -37 * a.max()
                    n_eps = 16 * np.sqrt(len(w)) * EPS
                    o[t, x] = a @ cc / l
                    bound[t, x] = (ea @ np.abs(cc) + n_eps * (a @ np.abs(cc))) / l + np.abs(
                        o[t, x]) * ((w @ rel) / l + n_eps)
            t += 1
    return o, bound + R._half_ulp(o, out)


def check(c, new, lengths, group, out, window=0, sinks=0, Q=None, seed=0):
    say(f"case: rows {c.kind} new={new} len={lengths} heads={c.heads} group={group} dim={c.dim} "
        f"page={c.page} window={window} sinks={sinks} {out}")
    c.device()
    n_tok, H = sum(new), c.heads * group
    if Q is None:
        Q = 2 * np.random.default_rng(seed + 5).standard_normal((n_tok, H * c.dim))
    Q = Q.astype(np.float16)
    got = B.kv8_attention(c.kv, torch.from_numpy(Q).to(DEV),
                          ints(np.concatenate([[0], np.cumsum(new)])), ints(lengths), c.tab, H,
                          window=window, sinks=sinks, odtype=OUT[out])
    torch.cuda.synchronize()
    got = got.double().cpu().numpy().reshape(n_tok, H, c.dim)
    ref, bound = row_reference(c, Q.astype(np.float64), new, lengths, group, window, sinks, out)
    nan = np.isnan(ref)
    assert (np.isnan(got) == nan).all(), (
        "NaN where the row sees none, or none where it sees one",
        np.argwhere(np.isnan(got) != nan)[:4].tolist())
    over = np.where(nan, -1.0, np.abs(got - ref) - bound)
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, (at, got[at], ref[at], bound[at])
    return got


# few rows share the keys between the waves, many have them each for itself
SHAPES = [([9], [70], 1), ([5], [50], 4), ([96], [96], 1), ([70, 33], [130, 33], 2)]


def steps(c, lengths, exponents):
    """Value scales of a request's pages in order: 2^(exponents[i]) times about one."""
    for r, n in enumerate(lengths):
        for i in range(-(-n // c.page)):
            c.vs[c.table[r, i]] = np.float32(2.0 ** exponents[min(i, len(exponents) - 1)] * 1.37)


# ------------------------------------------------------------------------------- value scales

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lengths,group", SHAPES)
@pytest.mark.parametrize("step", [12, 24, 34])
def test_large_scales_of_later_pages(kind, new, lengths, group, step):
    """Each page's values are 2^step times the page's before: a row that ends in a page is worked
    on beside rows that see the next one."""
    c = Cache(np.random.default_rng(step), kind, 2, 64, 16, lengths)
    steps(c, lengths, [-60 + min(step * i, 102) for i in range(9)])
    check(c, new, lengths, group, "f32")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lengths,group", SHAPES)
def test_large_scales_that_a_window_leaves(kind, new, lengths, group):
    """Early pages of large values that later rows of a wave see no more."""
    c = Cache(np.random.default_rng(3), kind, 2, 128, 16, lengths)
    steps(c, lengths, [40 - 24 * i if i < 4 else -50 for i in range(9)])
    for window in (3, 20):
        check(c, new, lengths, group, "f32", window=window)


@pytest.mark.parametrize("new,lengths,group", SHAPES)
def test_large_scales_of_small_weights(new, lengths, group):
    """Keys of large value scales and softmax weights of about e^-40: their contributions are
    below, near and above the others'."""
    for ratio in (30, 58, 80):
        c = Cache(np.random.default_rng(ratio), "int8", 1, 64, 16, lengths)
        for r, n in enumerate(lengths):
            for i in range(-(-n // 16)):
                pg, far = c.table[r, i], i % 2
                c.k[pg] = np.int8(-60 if far else 40).view(np.uint8)
                c.ks[pg] = 1.0 / 20
                c.vs[pg] = np.float32(2.0 ** (ratio - 45 if far else -45))
        # s = 8 x 0.05 x (40 or -60): a difference of 40
        check(c, new, lengths, group, "f32", Q=np.ones((sum(new), group * 64)))


@pytest.mark.parametrize("new,lengths,group", SHAPES)
def test_zero_scales_of_large_weights(new, lengths, group):
    """Pages of values 0 that take nearly all of the softmax weight, or nearly none."""
    for zero in (0, 1):
        c = Cache(np.random.default_rng(4), "int8", 1, 64, 16, lengths)
        for r, n in enumerate(lengths):
            for i in range(-(-n // 16)):
                pg = c.table[r, i]
                c.k[pg] = np.int8(-60 if i % 2 else 40).view(np.uint8)
                c.ks[pg] = 1.0 / 50            # s = 6.4 or -9.6
                c.vs[pg] = 0.0 if i % 2 == zero else 0.3
        check(c, new, lengths, group, "f32", Q=np.ones((sum(new), group * 64)))


def test_scales_at_the_ends_of_fp32():
    for new, lengths, group in SHAPES:
        c = Cache(np.random.default_rng(8), "fp8", 2, 64, 16, lengths)
        steps(c, lengths, [-110, -20, 110, -110])
        check(c, new, lengths, group, "f32")


# ------------------------------------------------------------------------------- f16 output

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lengths,group", [
    ([1] * 90, [150 + 2 * r for r in range(90)], 2), ([3] * 20, [200 + r for r in range(20)], 4),
    ([64], [200], 2), ([200, 90], [330, 90], 1)])
def test_f16_output_has_only_its_own_rounding(kind, new, lengths, group):
    """The weights keep two f16 values where the output is f16 too.  With one, a weight errs by up
    to 2^-12 of itself, and over values of both signs the sum by as much as the output's rounding:
    together 1.4 times that in the mean.  With two, nothing else comes near 2^-14."""
    c = Cache(np.random.default_rng(6), kind, 2, 128, 64, lengths)
    Q = np.random.default_rng(7).standard_normal((sum(new), 2 * group * 128)).astype(np.float16)
    got = check(c, new, lengths, group, "f16", Q=Q)
    ref, _ = row_reference(c, Q.astype(np.float64), new, lengths, group, 0, 0, "f16")
    rms = lambda e: float(np.sqrt((e ** 2).mean()))  # noqa: E731
    assert rms(got - ref) <= 1.1 * rms(ref.astype(np.float16).astype(np.float64) - ref)


# ------------------------------------------------------------------------------- NaN

def places(lengths):
    """Positions near the end of the first request, in pages that only some of its rows see."""
    n = lengths[0]
    return sorted({n - 1, n - 2, n - 4, max(n - 20, 0), 3})


@pytest.mark.parametrize("new,lengths,group", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
def test_nan_value_codes(new, lengths, group, page):
    """A NaN code of V makes NaN of its dim for the rows that see its key, and of nothing else."""
    for window, sinks in ((0, 0), (7, 2)):
        c = Cache(np.random.default_rng(1), "fp8", 2, 96, page, lengths)
        for i, j in enumerate(places(lengths)):
            c.v[c.table[0, j // page], i % 2, 5 + 17 * i, j % page] = 0x7F if i % 3 else 0xFF
        got = check(c, new, lengths, group, "f32", window=window, sinks=sinks)
        assert np.isnan(got).any() and not np.isnan(got).all(-1).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,lengths,group", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
def test_nan_scales(kind, new, lengths, group, page):
    """A page's NaN scale, of K or V, makes NaN of the rows that see a key of it, and of no other."""
    for which in ("ks", "vs"):
        for window in (0, 5):
            for at in (0, (lengths[0] - 1) // page):
                c = Cache(np.random.default_rng(2), kind, 2, 64, page, lengths)
                getattr(c, which)[c.table[0, at], 1] = np.nan
                check(c, new, lengths, group, "f32", window=window)
