"""The plain forms that the GPU tests of pages and beams compare with, on cases worked out by hand."""
import numpy as np

from tests import pages_ref as R


def arr(*v):
    return np.array(v)


def test_tables_by_hand():
    refs = arr(1, 0, 2, 0, 0, 1)
    table = np.full((2, 4), -1)
    table[0, 0], table[1, 0] = 0, 5
    b = R.tables(refs, 16, [10, 16], [30, 1], 40, table)
    # request 0: tokens 10 .. 39 on entries 0, 1, 2; request 1: token 16 on entry 1
    assert table.tolist() == [[0, 1, 3, -1], [5, 4, -1, -1]]
    assert refs.tolist() == [1, 1, 2, 1, 1, 1]
    assert b["tok_start"].tolist() == [0, 30, 31] and b["length"].tolist() == [40, 17]
    assert b["slot"][0] == 10 and b["slot"][6] == 16 and b["slot"][29] == 3 * 16 + 7
    assert b["slot"][30] == 64 and b["tok_pos"][30] == 16 and b["tok_req"][30] == 1
    assert (b["slot"][31:] == -1).all() and (b["tok_req"][31:] == -1).all()
    assert b["missing"][0] == 0
    again = R.tables(refs, 16, [10, 16], [30, 1], 40, table)
    assert all((again[k] == b[k]).all() for k in b)
    # no page is free any more
    b = R.tables(refs, 16, [40, 17], [30, 0], 40, table)
    assert b["missing"][0] == 1 and table[0, 3] == -1 and b["slot"][8] == -1
    assert b["slot"][7] == 3 * 16 + 15


def test_release_by_hand():
    refs, table = arr(2, 1, 1), arr([0, 1, -1], [0, 7, 2])
    R.release(refs, table, first=[1, -3], last=[3, 2])
    assert refs.tolist() == [1, 0, 1] and table.tolist() == [[0, -1, -1], [-1, -1, 2]]
    R.release(refs, table)
    assert refs.tolist() == [0, 0, 0] and (table == -1).all()


def test_reorder_by_hand():
    # two beams of one prompt (page 0 shared), 20 tokens, own pages 1 and 2
    refs, table = arr(2, 1, 1, 0, 0), arr([0, 1, -1], [0, 2, -1])
    out, length, src, dst, missing = R.reorder(refs, 16, table, [20, 20], [1, 1])
    # page 1 is free again and is the lowest; row 0 keeps page 2
    assert out.tolist() == [[0, 2, -1], [0, 1, -1]] and refs.tolist() == [2, 1, 1, 0, 0]
    assert src.tolist() == [-1, 2] and dst.tolist() == [-1, 1] and missing[0] == 0
    # kept rows: nobody owns the page alone
    refs = arr(2, 1, 1, 0, 0)
    out, length, src, dst, missing = R.reorder(refs, 16, table, [20, 20], [1, 1], keep=True)
    assert out.tolist() == [[0, 3, -1], [0, 4, -1]] and refs.tolist() == [4, 1, 1, 1, 1]
    # pages that are full are shared, rows of no parent are empty
    refs = arr(2, 1, 1, 0, 0)
    out, length, src, dst, missing = R.reorder(refs, 16, table, [32, 20], [0, 0, -1, 5])
    assert out.tolist()[:2] == [[0, 1, -1]] * 2 and (out[2:] == -1).all()
    assert length.tolist() == [32, 32, 0, 0] and refs.tolist() == [2, 2, 0, 0, 0]


def test_beams_by_hand():
    logits = np.log(arr([0.5, 0.25, 0.25], [0.1, 0.2, 0.7]))
    parent, token, score, done, _ = R.beam_select(logits, [-1.0, -1.2], 2, eos=2)
    # -1 + log .5 = -1.69, -1.2 + log .7 = -1.56
    assert parent.tolist() == [1, 0] and token.tolist() == [2, 0] and done.tolist() == [True, False]
    np.testing.assert_allclose(score, [-1.2 + np.log(0.7), -1 + np.log(0.5)])
    parent, token, score, done, _ = R.beam_select(logits, [-np.inf, -1.2], 2, eos=1, done=[0, 1])
    assert parent.tolist() == [1, 0] and token.tolist() == [1, -1] and score[0] == -1.2
    parent, token, *_ = R.beam_select(np.zeros((2, 3)), [0.0, 0.0], 2)
    assert parent.tolist() == [0, 0] and token.tolist() == [0, 1]
