"""The float64 forms that the serving operators are tested against, on small cases worked out
otherwise: by hand, by the oracle's E4M3 codec, by a dense softmax."""
import numpy as np

import oracle as O
from tests import serving_ref as R


def test_e4m3_values_and_encoder():
    for c in range(256):
        if c & 0x7F != 0x7F:
            assert R.E4M3[c] == O.e4m3_value(c)
    rng = np.random.default_rng(0)
    x = np.concatenate([np.abs(rng.standard_normal(2000)) * 10.0 ** rng.integers(-4, 4, 2000),
                        R.E4M3[:127], (R.E4M3[:126] + R.E4M3[1:127]) / 2, [500.0, 1e9, 0.0]])
    x = x.astype(np.float32)
    got = R.encode(x, np.ones_like(x), "fp8")
    assert [int(c) for c in got] == [O.e4m3_nearest(float(v)) for v in x]
    assert (R.encode(-x[x > 0], np.ones(1, np.float32), "fp8") & 0x80).all()
    codes = R.encode(np.float32([1.5, 2.5, -2.5, 200, -200, 0.49]), np.float32([1]), "int8")
    assert codes.view(np.int8).tolist() == [2, 2, -2, 127, -127, 0]
    assert R.encode(np.float32([-3.0]), np.float32([0]), "fp8").tolist() == [0]


def test_adapter_by_hand():
    X = np.array([[1.0, 2.0], [3.0, -1.0], [1.0, 1.0]])
    A = np.array([[[1.0, 1.0], [0.0, 2.0]], [[5.0, 0.0], [9.0, 9.0]]])
    B = np.array([[[1.0, 2.0], [0.0, 1.0], [1.0, 0.0]], [[2.0, 7.0], [1.0, 7.0], [0.0, 7.0]]])
    base = np.full((3, 3), 10.0)
    y, bound = R.adapter(X, A, B, [2, 1], [0.5, 2.0], [0, 1, -1], base, "f32")
    # token 0: U = (3, 4), B U = (11, 4, 3); token 1: rank 1, U = 15, B U = (30, 15, 0)
    assert y.tolist() == [[15.5, 12.0, 11.5], [70.0, 40.0, 10.0], [10.0, 10.0, 10.0]]
    assert (bound > 0).all() and bound.max() < 1e-3


def _cache(kind, lengths, heads=2, dim=8, page=4):
    n = sum(-(-t // page) for t in lengths) + 1
    table = np.full((len(lengths), max(-(-t // page) for t in lengths)), -1, np.int32)
    at = 1
    for r, t in enumerate(lengths):
        for i in range(-(-t // page)):
            table[r, i] = at
            at += 1
    z = lambda *s: np.zeros(s, np.uint8)  # noqa: E731
    return (z(n, heads, page, dim), z(n, heads, dim, page), np.zeros((n, heads), np.float32),
            np.zeros((n, heads), np.float32), table)


def test_append_then_attention_equal_a_dense_softmax():
    """One token after the other and all at once give the same scales; attention over the decoded
    cache is a masked softmax."""
    rng = np.random.default_rng(1)
    for kind in ("fp8", "int8"):
        n, heads, dim, page = 11, 2, 8, 4
        K, V = rng.standard_normal((2, n, heads * dim)).astype(np.float32)
        one = _cache(kind, [n])
        R.append(*one[:4], kind, K, V, [0, n], [0], one[4], page)
        step = _cache(kind, [n])
        for t in range(n):
            R.append(*step[:4], kind, K[t:t + 1], V[t:t + 1], [0, 1], [t], step[4], page)
        np.testing.assert_array_equal(one[2], step[2])
        np.testing.assert_array_equal(one[3], step[3])
        top = 448 if kind == "fp8" else 127
        j = np.arange(n)
        pg = one[4][0, j // page]
        k = R.decode(one[0][pg, :, j % page], kind) * one[2][pg][:, :, None]
        v = R.decode(one[1][pg, :, :, j % page], kind) * one[3][pg][:, :, None]
        step8 = one[2][pg].max() * top / (8 if kind == "fp8" else 127)
        assert np.abs(k - K.reshape(n, heads, dim)).max() <= step8
        assert one[2][1, 0] == np.abs(K[:4, :8]).max() / np.float32(top)
        Q = rng.standard_normal((3, 4 * dim))
        for window, sinks in ((0, 0), (3, 0), (3, 2), (1, 1)):
            o, bound, written = R.attention(*one[:4], kind, Q, [0, 3], [n], one[4], 4, 0.3, window,
                                            sinks, "f32")
            assert written.all()
            for t in range(3):
                p = n - 3 + t
                see = (j <= p) & ((p - j < window) | (j < sinks) if window else True)
                for h in range(4):
                    s = np.where(see, k[:, h // 2] @ Q[t, h * dim:(h + 1) * dim] * 0.3, -np.inf)
                    w = np.exp(s - s.max())
                    np.testing.assert_allclose(o[t, h], w @ v[:, h // 2] / w.sum(), rtol=1e-12)


def test_attention_rows_that_see_nothing():
    c = _cache("fp8", [3])
    o, _, written = R.attention(*c[:4], "fp8", np.ones((5, 16)), [1, 5], [3], c[4], 2, 1.0, 0, 0,
                                "f16")
    assert not written[0] and written[1:].all() and (o == 0).all()


def test_append_values():
    c = _cache("int8", [4], heads=1)
    K = np.zeros((3, 8), np.float32)
    K[0, :3] = np.nan, np.inf, -1e30
    R.append(*c[:4], "int8", K, K, [0, 3], [0], c[4], 4)
    assert c[2][1, 0] == np.float32(65504) / np.float32(127)
    assert c[0][1, 0, 0].view(np.int8).tolist() == [0, 127, -127, 0, 0, 0, 0, 0]
    before = c[0].copy()
    R.append(*c[:4], "int8", K[1:2], K[1:2], [0, 1], [3], c[4], 4)    # a zero: the scale stays
    np.testing.assert_array_equal(before, c[0])
