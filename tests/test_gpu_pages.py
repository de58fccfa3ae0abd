"""Page tables, slot maps, rows given back, forked and reordered, and copied pages on the GPU
against the plain forms.  Whole numbers and codes: every value has to be equal."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import pages_ref as R
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def ints(v, dt=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(v)).to(dt).to(DEV)


def same(got, want, what):
    g = got.cpu().numpy()
    w = np.asarray(want).astype(g.dtype)
    assert g.shape == w.shape and np.array_equal(g, w), (what, np.flatnonzero(g.ravel() != w.ravel())[:8])


class Pool:
    """Random use of a pool, and rows that own some of its pages."""

    def __init__(self, rng, n_pages, page, cached, width, fill, kept=0):
        self.page, self.n = page, n_pages
        order = rng.permutation(n_pages)
        self.table = np.full((len(cached), width), -1)
        at = 0
        for r, c in enumerate(cached):
            m = min(-(-max(c, 0) // page) + (rng.integers(0, kept + 1) if kept else 0), width,
                    n_pages - at)
            self.table[r, :m] = order[at:at + m]
            at += m
        self.refs = np.zeros(n_pages, np.int64)
        self.refs[order[:at]] = 1
        rest = order[at:]
        self.refs[rest] = np.where(rng.random(len(rest)) < fill, rng.integers(1, 4, len(rest)), 0)

    def device(self, pad=0):
        """(refs, table) on the GPU; rows `pad` entries apart from each other."""
        wide = np.full((self.table.shape[0], self.table.shape[1] + pad), 99)
        wide[:, :self.table.shape[1]] = self.table
        return ints(self.refs), ints(wide)[:, :self.table.shape[1]]


CASES = [  # n_req, page, pool, cached, new, n_tok beyond the sum, fill
    (1, 64, 50, 0, 1, 0, 0.5), (1, 16, 7, 15, 1, 0, 0.0), (1, 16, 7, 16, 1, 0, 0.0),
    (3, 32, 64, 100, 40, 5, 0.3), (32, 64, 900, 1500, 1, 0, 0.5), (64, 128, 5000, 400, 3, 9, 0.9),
    (200, 16, 40000, 100, 60, -77, 0.6), (1023, 16, 70001, 40, 2, 11, 0.5),
    (1024, 32, 33000, 33, 4, 0, 0.95), (1025, 16, 99999, 20, 3, 100, 0.97),
    (2100, 16, 3000, 5, 1, 3, 0.2), (5, 16, 32768, 0, 4000, 0, 0.9), (2, 128, 32769, 0, 4097, 0, 1.0),
    (4, 16, 65537, 7, 9000, -1, 0.4)]


@pytest.mark.parametrize("n_req,page,pool,cached,new,beyond,fill", CASES)
def test_tables(n_req, page, pool, cached, new, beyond, fill):
    rng = np.random.default_rng(n_req * 7 + pool)
    c = rng.integers(0, cached + 1, n_req)
    n = rng.integers(0, new + 1, n_req)
    c[0], n[0] = cached, new
    if n_req > 2:
        c[1], n[2] = -5, -1
    n_tok = max(0, int(np.maximum(n, 0).sum()) + beyond)
    width = -(-int((np.maximum(c, 0) + np.maximum(n, 0)).max()) // page) + 2
    p = Pool(rng, pool, page, c, width, fill)
    refs, table = p.device(pad=3)
    say(f"case: tables n_req={n_req} page={page} pool={pool} n_tok={n_tok}")
    batch = B.kv8_tables(refs, page, ints(c), ints(n), table, n_tok=n_tok)
    want = R.tables(p.refs, page, c, n, n_tok, p.table)
    for name, w in want.items():
        same(getattr(batch, name), w, name)
    same(refs, p.refs, "refs")
    same(table, p.table, "table")
    # the same again changes nothing but what is still missing
    batch = B.kv8_tables(refs, page, ints(c), ints(n), table, batch)
    for name, w in want.items():
        same(getattr(batch, name), w, name)
    same(refs, p.refs, "refs again")
    same(table, p.table, "table again")


def test_tables_of_nothing():
    refs, table = ints(np.zeros(5)), ints(np.full((0, 4), -1))
    none = ints(np.zeros(0))
    b = B.kv8_tables(refs, 16, none, none, table, n_tok=9)
    assert b.tok_start.tolist() == [0] and b.missing.tolist() == [0]
    assert (b.tok_req == -1).all() and (b.tok_pos == -1).all() and (b.slot == -1).all()
    # requests, but no rows for their tokens; and no maps wanted
    b = B.DeviceBatch(ints(np.ones(3)), ints(np.ones(2)), None, None, None, ints([7]), 0)
    table = ints(np.full((2, 4), -1))
    B.kv8_tables(refs, 16, ints([3, 0]), ints([5, 6]), table, b)
    assert b.tok_start.tolist() == [0, 0, 0] and b.length.tolist() == [3, 0]
    assert b.missing.tolist() == [0] and not refs.any() and (table == -1).all()


def test_tables_past_the_row_and_odd_entries():
    """Positions behind the row's entries have no slot; entries that name no page are no page."""
    refs, table = np.array([1, 0, 0, 0]), np.array([[0, 77, -9]])
    r, t = ints(refs), ints(table)
    b = B.kv8_tables(r, 16, ints([16]), ints([60]), t, n_tok=60)
    want = R.tables(refs, 16, [16], [60], 60, table)
    for name, w in want.items():
        same(getattr(b, name), w, name)
    assert t.tolist() == [[0, 1, 2]] and b.missing.tolist() == [0] and b.slot[32:].max() == -1
    big = 2 ** 31 - 2           # the last positions there are
    b = B.kv8_tables(r, 16, ints([big]), ints([5]), t, n_tok=5)
    assert b.length.tolist() == [2 ** 31 - 1] and b.slot.max() == -1 and r.tolist() == [1, 1, 1, 0]


@pytest.mark.parametrize("rows,width", [(1, 1), (3, 300), (40, 77), (300, 2000)])
def test_release(rows, width):
    rng = np.random.default_rng(rows)
    table = rng.integers(-2, 5000, (rows, width))
    refs = R.counts(4000, table)
    first, last = rng.integers(-3, width + 3, rows), rng.integers(-3, width + 3, rows)
    for f, la in ((first, last), (None, first), (last, None), (None, None)):
        r, t = ints(refs), ints(table)
        say(f"case: release rows={rows} width={width} first={f is not None} last={la is not None}")
        B.kv8_release(r, t, None if f is None else ints(f), None if la is None else ints(la))
        wr, wt = refs.copy(), table.copy()
        R.release(wr, wt, f, la)
        same(r, wr, "refs")
        same(t, wt, "table")


def test_release_of_any_entries():
    """first and last are clamped to the row, whatever they are."""
    ends = [-2 ** 31, -1, 0, 299, 300, 301, 2 ** 31 - 300, 2 ** 31 - 1]
    first, last = (np.repeat(ends, 8), np.tile(ends, 8))
    table = np.arange(64 * 300).reshape(64, 300)
    refs = np.ones(64 * 300, np.int64)
    r, t = ints(refs), ints(table)
    B.kv8_release(r, t, ints(first), ints(last))
    R.release(refs, table, first, last)
    same(r, refs, "refs")
    same(t, table, "table")


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("n_in,n_out,page,length,width,spare", [
    (1, 1, 16, 5, 3, 0), (1, 4, 64, 777, 20, 9), (4, 4, 16, 100, 12, 3), (8, 8, 128, 2000, 30, 40),
    (13, 104, 32, 300, 25, 200), (104, 13, 32, 300, 25, 1), (1500, 1100, 16, 60, 7, 300),
    (6, 9, 16, 40, 2, 50), (5, 2000, 16, 33, 4, 3000),
    # at the ends of what one launch takes
    (1024, 1024, 16, 20, 2, 900), (1024, 1025, 16, 20, 2, 900), (1025, 1, 16, 20, 3, 5), (2, 2, 64, 900, 1024, 3),
    (2, 2, 64, 900, 1025, 3)])
def test_reorder(n_in, n_out, page, length, width, spare, keep):
    rng = np.random.default_rng(n_in * 31 + n_out)
    lens = rng.integers(-2, length + 1, n_in)
    lens[0] = length
    n_pages = n_in * width + spare
    # rows that share their first pages, as forks do, with pages past their length
    p = Pool(rng, n_pages, page, lens, width, 0.0, kept=2)
    for r in range(1, n_in, 3):
        full = min(max(int(lens[r]), 0), max(int(lens[r - 1]), 0)) // page
        p.table[r, :min(full, width)] = p.table[r - 1, :min(full, width)]
    others = rng.integers(0, n_pages, spare)       # held by a table that this call does not see
    p.refs = R.counts(n_pages, p.table, others)
    parent = rng.integers(-1, n_in + 1, n_out)
    parent[0] = 0
    refs, table = p.device(pad=1)
    out = ints(np.full((n_out, width + 5), 55))[:, :width]
    say(f"case: reorder {n_in}->{n_out} page={page} keep={keep}")
    got = B.kv8_reorder(refs, page, table, ints(lens), ints(parent), out, keep=keep)
    want = R.reorder(p.refs, page, p.table, lens, parent, keep)
    same(out, want[0], "table_out")
    for g, w, what in zip(got, want[1:], ("length_out", "src", "dst", "missing")):
        same(g, w, what)
    same(refs, p.refs, "refs")
    same(table, p.table, "table")                  # not written
    held = [p.table] if keep else []
    assert np.array_equal(p.refs, R.counts(n_pages, want[0], others, *held))


@pytest.mark.parametrize("kind,heads,dim,page,layers", [
    ("fp8", 2, 64, 16, 1), ("int8", 3, 96, 32, 3), ("fp8", 5, 128, 64, 2), ("int8", 1, 256, 128, 16)])
def test_copy_pages(kind, heads, dim, page, layers):
    rng = np.random.default_rng(page)
    n = 12
    kvs, host = [], []
    for _ in range(layers):
        h = [rng.integers(0, 256, (n, heads, page, dim)).astype(np.uint8),
             rng.integers(0, 256, (n, heads, dim, page)).astype(np.uint8),
             rng.random((n, heads)).astype(np.float32), rng.random((n, heads)).astype(np.float32)]
        host.append(h)
        kvs.append(B.DeviceKV8(*[torch.from_numpy(x.copy()).to(DEV) for x in h], kind))
    src, dst = np.array([3, -1, 3, 4, 0, 12, 5]), np.array([7, 8, 2, 4, -1, 6, 11])
    for length in (None, np.array([1, 5, 16, 3, 9, 2, page]),
                   np.array([page + 17, 5, 2 * page - 1, 3, 9, 2, -3])):
        say(f"case: copy {kind} heads={heads} dim={dim} page={page} length={length is not None}")
        B.kv8_copy_pages(kvs, ints(src), ints(dst), None if length is None else ints(length))
        for kv, h in zip(kvs, host):
            R.copy_pages(*h, src, dst, length)
            for t, w in zip((kv.k, kv.v, kv.kscale, kv.vscale), h):
                same(t, w, "cache")


@pytest.mark.parametrize("width", [3, 5000])
def test_reorder_of_nothing_and_to_nothing(width):
    """No rows before, none after; in one launch and in two."""
    none = ints(np.zeros(0))
    table = np.full((3, width), -1)
    table[:, :3] = np.arange(9).reshape(3, 3)
    refs, out = ints([1] * 9 + [0]), ints(np.full((3, width), 7))
    got = B.kv8_reorder(refs, 16, ints(np.zeros((0, width))), none, ints([0, -1, 5]), out)
    assert (out == -1).all() and [t.tolist() for t in got] == [[0] * 3, [-1] * 3, [-1] * 3, [0]]
    assert refs.tolist() == [1] * 9 + [0]
    got = B.kv8_reorder(refs, 16, ints(table), ints([40, 48, 0]), none, ints(np.zeros((0, width))))
    assert not refs.any() and [t.tolist() for t in got] == [[], [], [], [0]]


def test_copies_past_32_bits():
    """Caches of more than 4 GiB: pages at either end, and between them."""
    say("case: copies over 4 GiB")
    n, heads, dim, page = 33000, 8, 128, 128
    kv = B.DeviceKV8.empty(n, heads, dim, page, "int8", DEV)
    assert kv.k.numel() > 2 ** 32
    rng = np.random.default_rng(3)
    src, dst = [0, n - 1, 17000, 5], [n - 2, 1, n - 3, 32900]
    want = []
    for s in src:
        for t in (kv.k, kv.v):
            t[s] = torch.from_numpy(rng.integers(0, 256, t[s].shape).astype(np.uint8)).to(DEV)
        kv.kscale[s] = torch.from_numpy(rng.random(heads).astype(np.float32)).to(DEV)
        kv.vscale[s] = torch.from_numpy(rng.random(heads).astype(np.float32)).to(DEV)
        want.append([t[s].clone() for t in (kv.k, kv.v, kv.kscale, kv.vscale)])
    B.kv8_copy_pages([kv], ints(src), ints(dst))
    for s, d, w in zip(src, dst, want):
        for t, x in zip((kv.k, kv.v, kv.kscale, kv.vscale), w):
            assert torch.equal(t[s], x) and torch.equal(t[d], x)
