"""GPU parity of the serving operators (adapters beside a projection, the 8-bit key/value cache
and attention over it) with their float64 forms: element types, odd sizes, strides, lengths of
zero and one, rows that see nothing, missing pages, garbage in unused places, streams, capture."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import serving_ref as R
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
OUT = {"f16": torch.float16, "f32": torch.float32}
KINDS = ("fp8", "int8")


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device=DEV)


def within(y, ref, bound, what):
    y = y.detach().double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(y).all(), f"{what}: not finite"
    over = np.abs(y - ref) - bound
    assert (over <= 0).all(), (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))


# ------------------------------------------------------------------------------- adapters

def make_adapters(rng, n, r_max, d_in, d_out, ranks, pad=0):
    """Random adapters; what the ranks leave unused holds NaN."""
    r8, c8 = -(-r_max // 8) * 8 + pad, -(-d_in // 8) * 8 + pad
    A = np.full((n, r_max, c8), np.nan, np.float16)
    Bm = np.full((n, d_out, r8), np.nan, np.float16)
    for a in range(n):
        r = min(max(int(ranks[a]), 0), r_max)
        A[a, :r, :d_in] = rng.standard_normal((r, d_in)) / np.sqrt(d_in)
        Bm[a, :, :r] = rng.standard_normal((d_out, r)) * 0.3
    scale = (rng.standard_normal(n) + 2).astype(np.float32)
    ad = B.DeviceAdapters(torch.from_numpy(A).to(DEV)[:, :, :d_in], torch.from_numpy(Bm).to(DEV),
                          ints(ranks), torch.from_numpy(scale).to(DEV), r_max=r_max)
    clean = lambda t: np.nan_to_num(t.astype(np.float64))  # noqa: E731
    return ad, (clean(A[:, :, :d_in]), clean(Bm[:, :, :r_max]), np.asarray(ranks), scale)


def check_adapter(T, n, r_max, d_in, d_out, out, ranks, ids, base="given", pad=0, seed=0):
    say(f"case: adapters T={T} n={n} r_max={r_max} {d_in}->{d_out} {out} base={base} pad={pad}")
    rng = np.random.default_rng(seed + 7 * T + d_in)
    ad, ref = make_adapters(rng, n, r_max, d_in, d_out, ranks, pad)
    X = torch.full((T, -(-d_in // 8) * 8 + pad), float("nan"), dtype=torch.float16, device=DEV)
    X = X[:, :d_in]
    X.copy_(torch.from_numpy(rng.standard_normal((T, d_in)).astype(np.float16)))
    b = torch.from_numpy(rng.standard_normal((T, d_out + pad)).astype(np.float32)).to(DEV)
    b = b.to(OUT[out])[:, :d_out]
    before = None if base == "none" else b.double().cpu().numpy().copy()
    Y = b if base == "place" else torch.full((T, d_out + 2 * pad), float("nan"), dtype=OUT[out],
                                             device=DEV)[:, :d_out]
    got = B.dict_adapter_forward(X, ad, ints(ids), base=None if base == "none" else b, Y=Y)
    torch.cuda.synchronize()
    y, bound = R.adapter(X.double().cpu().numpy(), *ref, ids, before, out)
    within(got, y, bound, "adapters")
    if base == "given":
        again = B.dict_adapter_forward(X, ad, ints(ids), base=b, ydtype=OUT[out])
        assert torch.equal(again, got)


@pytest.mark.parametrize("T,n,r_max,d_in,d_out,out,pad", [
    (1, 1, 16, 256, 128, "f16", 0), (1, 3, 1, 8, 1, "f32", 0), (2, 4, 16, 4096, 1024, "f16", 0),
    (5, 2, 64, 1000, 333, "f32", 8), (16, 16, 8, 520, 1029, "f16", 0),
    (17, 3, 33, 777, 250, "f16", 16), (64, 5, 128, 512, 512, "f32", 0),
    (100, 40, 256, 264, 100, "f16", 0), (257, 4, 20, 640, 320, "f32", 0),
    (1030, 7, 32, 328, 264, "f16", 8)])
def test_adapter_shapes(T, n, r_max, d_in, d_out, out, pad):
    rng = np.random.default_rng(T)
    ranks = [max(1, (r_max, r_max // 2, r_max - 1, 1)[i % 4]) for i in range(n)]
    ids = rng.integers(-1, n, T)
    ids[0] = n - 1
    check_adapter(T, n, r_max, d_in, d_out, out, ranks, ids, pad=pad)


@pytest.mark.parametrize("T", [1, 33, 300])
@pytest.mark.parametrize("base", ["given", "none", "place"])
def test_adapter_base_and_ids(T, base):
    rng = np.random.default_rng(3)
    for ids in (np.full(T, -1), np.full(T, 2), np.where(rng.random(T) < 0.5, 10 ** 6, 1),
                np.full(T, -2 ** 31), np.repeat([0, 3, 1], T)[:T]):
        check_adapter(T, 4, 24, 200, 190, "f16", [24, 0, 9, 99], ids, base=base)


def test_adapter_long_rows_and_many_tokens():
    rng = np.random.default_rng(5)
    check_adapter(3, 2, 128, 11008, 96, "f32", [128, 127], [1, 0, 1])
    ids = np.repeat(rng.integers(-1, 9, 40), rng.integers(1, 120, 40))
    check_adapter(len(ids), 9, 16, 96, 72, "f16", [16, 3, 8, 16, 1, 16, 12, 5, 16], ids)
    check_adapter(1100, 1100, 8, 64, 24, "f32", [8] * 1100, rng.permutation(1100))


@pytest.mark.parametrize("n", [3, 700, 2500])
def test_adapter_very_many_tokens(n):
    rng = np.random.default_rng(n)
    ranks = rng.integers(0, 9, n)
    for ids in (rng.integers(-1, n, 8300), np.repeat(rng.integers(-1, n, 30), 280)[:8193]):
        check_adapter(len(ids), n, 8, 40, 24, "f32", ranks, ids)


@pytest.mark.parametrize("r_max", [12, 27, 64, 70])
@pytest.mark.parametrize("T,n", [(300, 1), (1000, 3), (1000, 12), (9000, 5)])
def test_adapter_many_tokens_of_few_adapters(T, n, r_max):
    rng = np.random.default_rng(T + n + r_max)
    ranks = [max(1, r_max - 5 * i) for i in range(n)]
    ids = np.repeat(rng.integers(-1, n, T // 50 + 1), 50)[:T]
    check_adapter(T, n, r_max, 136, 200, "f16", ranks, ids)


@pytest.mark.parametrize("d_in", [2048, 2056, 4096, 4104])
@pytest.mark.parametrize("r_max", [16, 32])
def test_adapter_few_tokens_over_longer_rows(d_in, r_max):
    check_adapter(7, 3, r_max, d_in, 320, "f32", [r_max, 5, r_max - 1], [2, 0, -1, 1, 2, 2, 0])


def test_adapter_large_and_small_products():
    """X A^T far outside f16's range, and far below it."""
    rng = np.random.default_rng(4)
    ad, ref = make_adapters(rng, 2, 16, 256, 64, [16, 13])
    for size in (2.0 ** 9, 2.0 ** -22):
        X = (rng.standard_normal((18, 256)) * size).astype(np.float16)
        big = B.DeviceAdapters(ad.A * 64, ad.B, ad.rank, ad.scale, r_max=16) if size > 1 else ad
        want = (ref[0] * (64 if size > 1 else 1),) + ref[1:]
        ids = np.arange(18) % 2
        y = B.dict_adapter_forward(torch.from_numpy(X).to(DEV), big, ints(ids),
                                   ydtype=torch.float32)
        torch.cuda.synchronize()
        ref_y, bound = R.adapter(X, *want, ids, None, "f32")
        within(y, ref_y, bound, f"products of size {size}")


def test_adapter_small_ranks_beside_large_ones():
    """Ranks far below r_max, after a call that leaves NaN in the LDS of every CU."""
    rng = np.random.default_rng(6)
    ids = rng.integers(0, 3, 700)
    ad, _ = make_adapters(rng, 3, 64, 256, 512, [64, 64, 64])
    for T in (40, 700):
        X = torch.full((T, 256), float("nan"), dtype=torch.float16, device=DEV)
        B.dict_adapter_forward(X, ad, ints(ids[:T]))
        check_adapter(T, 3, 64, 96, 512, "f16", [1, 3, 40], ids[:T])
        check_adapter(T, 3, 256, 96, 128, "f32", [1, 17, 255], ids[:T])


def test_adapter_no_tokens():
    rng = np.random.default_rng(1)
    ad, _ = make_adapters(rng, 1, 8, 64, 32, [8])
    y = B.dict_adapter_forward(torch.empty(0, 64, dtype=torch.float16, device=DEV), ad, ints([]))
    assert y.shape == (0, 32)


def test_adapter_input_values():
    """Infinities and NaN of one token's row stay in that row."""
    rng = np.random.default_rng(2)
    ad, ref = make_adapters(rng, 2, 16, 128, 64, [16, 16])
    X = rng.standard_normal((20, 128)).astype(np.float16)
    bad = X.copy()
    bad[3, 5], bad[11, 7] = np.inf, np.nan
    ids = np.arange(20) % 2
    y = B.dict_adapter_forward(torch.from_numpy(bad).to(DEV), ad, ints(ids), ydtype=torch.float32)
    torch.cuda.synchronize()
    want, bound = R.adapter(X, *ref, ids, None, "f32")
    rows = [t for t in range(20) if t not in (3, 11)]
    within(y[rows], want[rows], bound[rows], "rows without a bad value")
    assert not torch.isfinite(y[3]).any() and torch.isnan(y[11]).all()


# ------------------------------------------------------------------------------- cache

class Cache:
    """A cache on the device and its numpy copy.  Unused slots and pages hold random bytes
    (NaN codes among them) and NaN scales."""

    def __init__(self, rng, kind, heads, dim, page, lengths, spare=3, cols=None, spread=False):
        self.kind, self.page, self.heads, self.dim = kind, page, heads, dim
        need = [-(-t // page) for t in lengths]
        n = sum(need) + spare
        order = rng.permutation(n)
        self.table = np.full((len(lengths), cols or max(max(need, default=0), 1)), -1, np.int32)
        self.k = rng.integers(0, 256, (n, heads, page, dim), np.uint8)
        self.v = rng.integers(0, 256, (n, heads, dim, page), np.uint8)
        self.ks = np.full((n, heads), np.nan, np.float32)
        self.vs = np.full((n, heads), np.nan, np.float32)
        at = 0
        for r, t in enumerate(lengths):
            for i in range(need[r]):
                pg = order[at]
                at += 1
                if i < self.table.shape[1]:
                    self.table[r, i] = pg
                m = min(page, t - i * page)
                for c, s in ((self.k[pg], self.ks), (self.v[pg].transpose(0, 2, 1), self.vs)):
                    x = rng.standard_normal((heads, m, dim)).astype(np.float32)
                    if spread:
                        x *= np.float32(10.0 ** rng.integers(-6, 4))
                    sc = np.abs(x).max((1, 2)) / np.float32(448 if kind == "fp8" else 127)
                    s[pg] = sc
                    c[:, :m] = R.encode(x, sc[:, None, None], kind)
        self.device()

    def device(self):
        t = lambda a: torch.from_numpy(a.copy()).to(DEV)  # noqa: E731
        self.kv = B.DeviceKV8(t(self.k), t(self.v), t(self.ks), t(self.vs), self.kind)
        self.tab = t(self.table)


def check_attention(c, new, lengths, group, out, window=0, sinks=0, pad=0, seed=0, scale=None,
                    starts=None, n_tok=None):
    say(f"case: attention {c.kind} new={list(new)[:8]} len={list(lengths)[:8]} heads={c.heads}"
        f" group={group} dim={c.dim} page={c.page} window={window} sinks={sinks} {out}")
    rng = np.random.default_rng(seed + 11)
    start = np.concatenate([[0], np.cumsum(new)]) if starts is None else np.asarray(starts)
    n_tok = int(start[-1]) if n_tok is None else n_tok
    H = c.heads * group
    Q = torch.full((n_tok, H * c.dim + pad), float("nan"), dtype=torch.float16, device=DEV)
    Q = Q[:, :H * c.dim]
    Q.copy_(torch.from_numpy((2 * rng.standard_normal((n_tok, H * c.dim))).astype(np.float16)))
    O = torch.full((n_tok, H * c.dim + pad), 77.0, dtype=OUT[out], device=DEV)[:, :H * c.dim]
    ws = B.kv8_attention_workspace(c.kv, len(lengths), n_tok, H, DEV)
    B.kv8_attention(c.kv, Q, ints(start), ints(lengths), c.tab, H, sm_scale=scale, window=window,
                    sinks=sinks, O=O, ws=ws)
    torch.cuda.synchronize()
    assert not ws[:65536].any(), "the first 64 KiB of the workspace are left zero"
    ref, bound, written = R.attention(c.k, c.v, c.ks, c.vs, c.kind, Q.double().cpu().numpy(), start,
                                      lengths, c.table, H, scale or c.dim ** -0.5, window, sinks,
                                      out)
    got = O.reshape(n_tok, H, c.dim)
    within(got[torch.from_numpy(written).to(DEV)], ref[written], bound[written], "attention")
    assert (got[torch.from_numpy(~written).to(DEV)] == 77.0).all(), "rows of no request"
    again = torch.empty_like(O)
    B.kv8_attention(c.kv, Q, ints(start), ints(lengths), c.tab, H, sm_scale=scale, window=window,
                    sinks=sinks, O=again, ws=ws)
    w = torch.from_numpy(written).to(DEV)
    assert torch.equal(again[w], O[w])
    return O


LENGTHS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 333, 700]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_attention_decode_lengths(kind, page, dim):
    rng = np.random.default_rng(page + dim)
    c = Cache(rng, kind, 2, dim, page, LENGTHS)
    check_attention(c, [1] * len(LENGTHS), LENGTHS, 1 + page // 32, "f16" if dim != 96 else "f32")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 3, 4, 5, 8, 16, 17])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_attention_groups_and_chunks(kind, group, out):
    rng = np.random.default_rng(group)
    lengths, new = [5, 90, 300, 41, 0, 130], [5, 1, 37, 0, 0, 3]
    c = Cache(rng, kind, 2, 64, 32, lengths)
    check_attention(c, new, lengths, group, out, pad=8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (64, 4), (63, 70),
                                          (100, 16), (129, 200), (10 ** 6, 4), (2 ** 31 - 1, 3),
                                          (7, 2 ** 31 - 1), (-3, 5)])
def test_attention_window_and_sinks(kind, window, sinks):
    rng = np.random.default_rng(abs(window) % 1000 + sinks % 1000)
    lengths, new = [1, 300, 257, 64, 150], [1, 1, 90, 64, 2]
    c = Cache(rng, kind, 1, 64, 16, lengths)
    check_attention(c, new, lengths, 2, "f16", window=window, sinks=sinks)
    check_attention(c, new, lengths, 2, "f32", window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,page,new", [(128, 64, [200, 0, 333]), (64, 16, [129, 64, 65]),
                                          (256, 128, [70, 1, 150]), (96, 32, [100, 31, 260])])
def test_attention_prompts(kind, dim, page, new):
    rng = np.random.default_rng(dim)
    lengths = [new[0], 50, new[2] + 77] if new[1] == 0 else [new[0] + 5, new[1], new[2]]
    c = Cache(rng, kind, 2, dim, page, lengths)
    check_attention(c, new, lengths, 2, "f16")
    check_attention(c, new, lengths, 1, "f32", window=40, sinks=3)


def test_attention_rows_that_see_nothing():
    rng = np.random.default_rng(1)
    lengths, new = [3, 0, 20], [7, 4, 20]      # more queries than keys: some stand before 0
    c = Cache(rng, "fp8", 2, 64, 16, lengths)
    O = check_attention(c, new, lengths, 2, "f16")
    assert (O[:4] == 0).all() and (O[7:11] == 0).all() and (O[4:7] != 0).any()
    c.table[2, :] = -1
    c.table[0, 0] = 10 ** 9
    c.device()
    O = check_attention(c, new, lengths, 2, "f32")
    assert (O == 0).all()
    check_attention(c, [1, 1, 1], [-5, 0, 20], 3, "f16")
    # page 0 is missing, and the window reaches no further back than it
    check_attention(c, [1, 1, 1], [9, 8, 7], 1, "f16", window=4, sinks=2)


def test_attention_missing_pages_and_short_tables():
    rng = np.random.default_rng(4)
    lengths = [300, 170, 64]
    c = Cache(rng, "int8", 2, 128, 16, lengths)
    c.table[0, 2:9] = -1
    c.table[1, 10] = c.k.shape[0]
    c.device()
    for new in ([1, 1, 1], [40, 100, 3]):
        check_attention(c, new, lengths, 2, "f16")
        check_attention(c, new, lengths, 2, "f32", window=140, sinks=4)
    c = Cache(rng, "fp8", 1, 64, 16, [400, 90], cols=7)     # lengths past the table
    check_attention(c, [1, 3], [400, 90], 4, "f16")
    check_attention(c, [200, 90], [400, 90], 4, "f32")


def test_attention_rows_of_no_request():
    rng = np.random.default_rng(6)
    c = Cache(rng, "fp8", 2, 64, 32, [50, 60, 70])
    check_attention(c, [1, 1, 1], [50, 60, 70], 2, "f16", starts=[2, 3, 3, 6], n_tok=9)
    check_attention(c, [1, 1, 1], [50, 60, 70], 2, "f16", starts=[-4, 1, 30, 31], n_tok=20)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_attention_uneven_scales(kind, out):
    """Page scales that differ by ten powers of ten, pages of zeros, large scores."""
    rng = np.random.default_rng(8)
    lengths = [200, 333, 64]
    c = Cache(rng, kind, 2, 64, 16, lengths, spread=True)
    c.ks[c.table[0, 3]], c.vs[c.table[0, 4]], c.vs[c.table[1, 0]] = 0.0, 0.0, 0.0
    c.ks *= np.float32(1e-3)
    c.device()
    check_attention(c, [1, 1, 1], lengths, 3, out)
    check_attention(c, [60, 2, 64], lengths, 3, out)
    check_attention(c, [1, 1, 1], lengths, 1, out, scale=30.0)
    c.vs[:] = 0.0
    c.device()
    assert (check_attention(c, [1, 9, 1], lengths, 1, out) == 0).all()


def test_attention_many_requests():
    rng = np.random.default_rng(9)
    lengths = rng.integers(0, 90, 700)
    c = Cache(rng, "fp8", 1, 64, 16, lengths)
    check_attention(c, (lengths > 0).astype(int), lengths, 2, "f16")
    check_attention(c, np.minimum(lengths, rng.integers(0, 4, 700)), lengths, 8, "f16")


def test_attention_long_and_short_together():
    rng = np.random.default_rng(10)
    lengths = [20000, 3, 1, 900]
    c = Cache(rng, "int8", 2, 64, 64, lengths)
    check_attention(c, [1, 1, 1, 1], lengths, 2, "f16")
    check_attention(c, [1, 3, 1, 200], lengths, 2, "f16")
    check_attention(c, [2, 1, 0, 1], lengths, 2, "f32", window=3000, sinks=4)


def _big_cache(kind):
    # more than 2^32 bytes of codes: the last pages lie past any 32-bit offset
    heads, dim, page = 32, 128, 128
    n = (1 << 32) // (heads * dim * page) + 40
    k = torch.empty(n, heads, page, dim, dtype=torch.uint8, device=DEV)
    v = torch.empty(n, heads, dim, page, dtype=torch.uint8, device=DEV)
    s = lambda: torch.empty(n, heads, dtype=torch.float32, device=DEV)  # noqa: E731
    return B.DeviceKV8(k, v, s(), s(), kind)


@pytest.mark.parametrize("kind", KINDS)
def test_cache_past_32_bit_offsets(kind):
    say(f"case: cache of more than 2^32 bytes, {kind}")
    rng = np.random.default_rng(12)
    big = _big_cache(kind)
    n = big.n_pages
    small = B.DeviceKV8.empty(4, big.heads, big.head_dim, big.page, kind, DEV)
    K, V = (torch.from_numpy(rng.standard_normal((450, 32 * 128)).astype(np.float16)).to(DEV)
            for _ in range(2))
    start, zero, length = ints([0, 450]), ints([0]), ints([450])
    ta, tb = ints([[n - 1, 0, n - 2, n - 3]]), ints([[3, 0, 2, 1]])
    Q = torch.from_numpy(rng.standard_normal((3, 32 * 128)).astype(np.float16)).to(DEV)
    outs = []
    for kv, t in ((big, ta), (small, tb)):
        B.kv8_append(kv, K, V, start, zero, t)
        outs.append(B.kv8_attention(kv, Q, ints([0, 3]), length, t, 32, odtype=torch.float32))
    torch.cuda.synchronize()
    assert torch.equal(big.k[n - 1], small.k[3]) and torch.equal(big.v[n - 3, :, :, :60],
                                                                 small.v[1, :, :, :60])
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()


# ------------------------------------------------------------------------------- append

def check_append(kind, heads, dim, page, cached, new, src="f16", pad=0, seed=0, edit=None,
                 table=None, starts=None, n_tok=None):
    say(f"case: append {kind} cached={list(cached)[:8]} new={list(new)[:8]} heads={heads} dim={dim}"
        f" page={page} {src}")
    rng = np.random.default_rng(seed + page)
    total = [max(a, 0) + b for a, b in zip(cached, new)]
    c = Cache(rng, kind, heads, dim, page, total)
    if table is not None:
        table(c)
        c.device()
    start = np.concatenate([[0], np.cumsum(new)]) if starts is None else np.asarray(starts)
    n_tok = int(start[-1]) if n_tok is None else n_tok
    dt = OUT[src]
    KV = []
    for i in range(2):
        x = torch.full((n_tok, heads * dim + pad), float("nan"), dtype=dt, device=DEV)
        x = x[:, :heads * dim]
        y = rng.standard_normal((n_tok, heads * dim)) * np.exp(rng.standard_normal((n_tok, 1)))
        if edit is not None:
            edit(y)
        x.copy_(torch.from_numpy(y.astype(np.float32)).to(dt))
        KV.append(x)
    k, v, ks, vs = (a.copy() for a in (c.k, c.v, c.ks, c.vs))
    R.append(k, v, ks, vs, kind, *(x.float().cpu().numpy() for x in KV), start, cached, c.table,
             page)
    B.kv8_append(c.kv, *KV, ints(start), ints(cached), c.tab)
    torch.cuda.synchronize()
    for got, want, what in ((c.kv.kscale, ks, "kscale"), (c.kv.vscale, vs, "vscale")):
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint32), want.view(np.uint32), what)
    for got, want, what in ((c.kv.k, k, "k"), (c.kv.v, v, "v")):
        np.testing.assert_array_equal(got.cpu().numpy(), want, what)
    # the same call again leaves the cache as it is
    B.kv8_append(c.kv, *KV, ints(start), ints(cached), c.tab)
    np.testing.assert_array_equal(c.kv.k.cpu().numpy(), k)
    np.testing.assert_array_equal(c.kv.vscale.cpu().numpy().view(np.uint32), vs.view(np.uint32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_append_shapes(kind, page, dim):
    check_append(kind, 3, dim, page, [0, 1, 15, 16, 100, 127, 128], [1, 1, 1, 1, 1, 1, 1])
    check_append(kind, 2, dim, page, [0, 5, 64, 31, 17], [300, 0, 65, 1, 40], src="f32", pad=5)


@pytest.mark.parametrize("kind", KINDS)
def test_append_values(kind):
    """Zeros, subnormals, NaN, infinities, values past f16's range, ties between codes."""
    def edit(y):
        y[0:3] = 0.0
        y[4, ::3], y[4, 1::3] = np.nan, np.inf
        y[5] = -np.inf
        y[6] = np.nan
        y[7] = 1e-7
        y[8] = -0.0
        y[9, :] = np.arange(y.shape[1]) / 16
        y[10, :] = 448.0 * np.sign(y[10, :])
        y[11, :] = np.linspace(-127, 127, y.shape[1])
        y[12] = 1e30
    for src in ("f16", "f32"):
        check_append(kind, 1, 128, 16, [3, 0, 9], [8, 8, 4], src=src, edit=edit)
        check_append(kind, 1, 64, 16, [0] * 20, [1] * 20, src=src, edit=edit)


def test_append_zero_page_then_values():
    """A page of zeros has scale 0; later values set it."""
    def edit(y):
        y[:] = 0.0
        y[-1] = np.arange(y.shape[1]) / 7
    for kind in KINDS:
        check_append(kind, 2, 64, 32, [0], [9], edit=edit)
        check_append(kind, 2, 64, 32, [7], [1], edit=lambda y: y.fill(0.0))


def test_append_tables_and_rows():
    def holes(c):
        c.table[0, 1] = -1
        c.table[1, 0] = c.k.shape[0]
        c.table = c.table[:, :4].copy()
    check_append("fp8", 2, 64, 16, [3, 5, 40], [60, 30, 60], table=holes)
    check_append("int8", 2, 64, 16, [-7, 5, 0], [20, 3, 0], src="f32")
    check_append("fp8", 1, 64, 32, [0, 9, 0], [4, 9, 2], starts=[3, 7, 7, 9], n_tok=12)
    rng = np.random.default_rng(3)
    check_append("int8", 1, 64, 16, rng.integers(0, 50, 300), rng.integers(0, 3, 300))


# ------------------------------------------------------------------------------- streams, capture

def test_decode_step_on_a_stream_and_captured():
    """Append, then attention, on a side stream and replayed from a graph: the replays follow the
    lengths and inputs that the device tensors hold, with eager work between them."""
    rng = np.random.default_rng(20)
    heads, group, dim, page, req = 4, 2, 128, 16, 5
    first = np.array([0, 15, 16, 130, 400])
    steps = 6
    c = Cache(rng, "fp8", heads, dim, page, list(first + steps))
    mirror = Cache.__new__(Cache)
    mirror.__dict__.update(c.__dict__)
    mirror.device()
    K, V = (torch.zeros(req, heads * dim, dtype=torch.float16, device=DEV) for _ in range(2))
    Q = torch.zeros(req, heads * group * dim, dtype=torch.float16, device=DEV)
    start, cached, length = ints(np.arange(req + 1)), ints(first), ints(first + 1)
    O = torch.zeros(req, heads * group * dim, dtype=torch.float16, device=DEV)
    ws = B.kv8_attention_workspace(c.kv, req, req, heads * group, DEV)

    def step(kv, tab, O, ws):
        B.kv8_append(kv, K, V, start, cached, tab)
        B.kv8_attention(kv, Q, start, length, tab, heads * group, O=O, ws=ws, window=200, sinks=4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.kv, c.tab, O, ws)          # warm up, on a stream of its own
    side.synchronize()
    c.device()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c.kv, c.tab, O, ws)
    for i in range(steps):
        say(f"case: captured decode step {i}")
        for t in (K, V, Q):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float16)))
        cached.copy_(ints(first + i))
        length.copy_(ints(first + i + 1))
        graph.replay()
        want = torch.zeros_like(O)
        step(mirror.kv, mirror.tab, want, B.kv8_attention_workspace(c.kv, req, req, heads * group,
                                                                     DEV))
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.isfinite(O).all() and (O != 0).any()
        assert torch.equal(c.kv.k, mirror.kv.k) and torch.equal(c.kv.vscale.view(torch.int32),
                                                                mirror.kv.vscale.view(torch.int32))


def test_adapter_on_a_stream_and_captured():
    rng = np.random.default_rng(21)
    ad, ref = make_adapters(rng, 6, 32, 512, 384, [32, 8, 16, 32, 5, 32])
    X = torch.zeros(9, 512, dtype=torch.float16, device=DEV)
    Y = torch.zeros(9, 384, dtype=torch.float32, device=DEV)
    ids = ints([0] * 9)
    ws = B.adapter_workspace(9, ad, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.dict_adapter_forward(X, ad, ids, Y=Y, ws=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.dict_adapter_forward(X, ad, ids, Y=Y, ws=ws)
    for i in range(4):
        X.copy_(torch.from_numpy(rng.standard_normal(X.shape).astype(np.float16)))
        now = rng.integers(-1, 6, 9)
        ids.copy_(ints(now))
        graph.replay()
        torch.cuda.synchronize()
        want, bound = R.adapter(X.cpu().numpy(), *ref, now, None, "f32")
        within(Y, want, bound, f"replay {i}")
        eager = B.dict_adapter_forward(X, ad, ids, ydtype=torch.float32)
        assert torch.equal(eager, Y)
