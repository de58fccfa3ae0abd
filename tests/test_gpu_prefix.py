"""Attention of requests that share their first tokens against the float64 form of the attention
over each request's own table, with its bounds: what is read once for a group is added to the rest
of a row by fp32 operations, two more among those that the bounds count."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import serving_ref as R
from tests.gpu_helpers import DEV, say
from tests.test_gpu_serving import KINDS, OUT, Cache, ints, within
from tests.test_gpu_serving_rows import row_reference

pytestmark = pytest.mark.gpu


def shared_cache(rng, kind, heads, dim, page, groups, lengths, prefix, cols=None):
    """A cache whose rows name the group's first pages as far as prefix[g] tokens fill them."""
    c = Cache(rng, kind, heads, dim, page, lengths, cols=cols)
    for g, (r0, r1) in enumerate(zip(groups, groups[1:])):
        for r in range(r0 + 1, r1):
            m = min(prefix[g], lengths[r0], lengths[r]) // page
            c.table[r, :m] = c.table[r0, :m]
    c.device()
    return c


def check(c, new, lengths, group, out, groups, shared, window=0, sinks=0, pad=0, seed=0, scale=None,
          starts=None, n_tok=None, ws=None):
    say(f"case: prefix {c.kind} groups={list(groups)[:8]} shared={list(shared)[:8]} "
        f"new={list(new)[:8]} len={list(lengths)[:8]} heads={c.heads} group={group} dim={c.dim} "
        f"page={c.page} window={window} sinks={sinks} {out}")
    rng = np.random.default_rng(seed + 11)
    start = np.concatenate([[0], np.cumsum(new)]) if starts is None else np.asarray(starts)
    n_tok = int(start[-1]) if n_tok is None else n_tok
    H = c.heads * group
    Q = torch.full((n_tok, H * c.dim + pad), float("nan"), dtype=torch.float16, device=DEV)
    Q = Q[:, :H * c.dim]
    Q.copy_(torch.from_numpy((2 * rng.standard_normal((n_tok, H * c.dim))).astype(np.float16)))
    O = torch.full((n_tok, H * c.dim + pad), 77.0, dtype=OUT[out], device=DEV)[:, :H * c.dim]
    if ws is None:
        ws = B.kv8_prefix_attention_workspace(c.kv, len(lengths), n_tok, H, DEV)
        ws[65536:] = 0xFF
    args = (c.kv, Q, ints(start), ints(lengths), c.tab, ints(groups), ints(shared), H)
    kw = dict(sm_scale=scale, window=window, sinks=sinks, ws=ws)
    B.kv8_prefix_attention(*args, O=O, **kw)
    torch.cuda.synchronize()
    assert not ws[:65536].any(), "the first 64 KiB of the workspace are left zero"
    ref, bound, written = R.attention(c.k, c.v, c.ks, c.vs, c.kind, Q.double().cpu().numpy(), start,
                                      lengths, c.table, H, scale or c.dim ** -0.5, window, sinks,
                                      out)
    got = O.reshape(n_tok, H, c.dim)
    w = torch.from_numpy(written).to(DEV)
    within(got[w], ref[written], bound[written], "attention")
    assert (got[~w] == 77.0).all(), "rows of no request"
    again = torch.full_like(O, 5.0)
    B.kv8_prefix_attention(*args, O=again, **kw)
    assert torch.equal(again[w], O[w])
    return O


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_decode(kind, page, dim):
    """Groups of one to seven requests, prefixes of no tile to ten, requests beside any group."""
    rng = np.random.default_rng(page + dim)
    groups = [1, 2, 9, 9, 12]
    lengths = [70, 300, 400, 389, 385, 500, 384, 390, 700, 130, 129, 131, 5, 0]
    prefix = [200, 384, 50, 128]
    c = shared_cache(rng, kind, 2, dim, page, groups, lengths, prefix)
    check(c, [1] * 13 + [0], lengths, 1 + page // 32, "f16" if dim != 96 else "f32", groups,
          [p // page * page for p in prefix])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 3, 5, 8, 16, 17, 32])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_groups_of_heads_and_drafts(kind, group, out):
    """From few rows to many for a request and for a group: every form of the two lines."""
    rng = np.random.default_rng(group)
    lengths = [260, 256, 300, 270, 261, 64, 65, 200]
    for groups, new in (([0, 8], [1] * 8), ([0, 5, 8], [3, 1, 2, 1, 5, 1, 0, 1]),
                        ([0, 2, 4, 5, 8], [1] * 8), ([0, 1, 2, 3, 4, 5, 6, 7, 8], [1] * 8)):
        c = shared_cache(rng, kind, 2, 64, 32, groups, lengths, [256] * 8)
        check(c, new, lengths, group, out, groups, [256, 192, 256, 64, 256, 64, 0, 256][:len(groups) - 1],
              pad=8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (64, 4), (63, 70),
                                          (150, 16), (170, 200), (10 ** 6, 4), (2 ** 31 - 1, 3),
                                          (7, 2 ** 31 - 1), (-3, 5)])
def test_window_and_sinks(kind, window, sinks):
    """Rows whose windows reach into the shared keys, only past them, or over all of them."""
    rng = np.random.default_rng(abs(window) % 1000 + sinks % 1000)
    lengths, new = [260, 330, 200, 450, 257, 90, 128], [1, 3, 1, 2, 1, 1, 1]
    groups = [0, 5, 7]
    c = shared_cache(rng, kind, 1, 64, 16, groups, lengths, [192, 64])
    for out, group in (("f16", 2), ("f32", 9)):
        check(c, new, lengths, group, out, groups, [192, 64], window=window, sinks=sinks)


def test_shared_of_any_size():
    """Shared tokens that are no whole page or tile, none, negative, past the requests' lengths and
    past the table."""
    rng = np.random.default_rng(21)
    lengths = [200, 210, 190, 220]
    for page in (16, 128):
        c = shared_cache(rng, "fp8", 2, 64, page, [0, 4], lengths, [190])
        for shared in (0, -7, 1, 63, 64, 100, 127, 128):
            check(c, [1] * 4, lengths, 2, "f16", [0, 4], [shared])
    # the same tokens all along: requests of 100, 130, 190 and 256 tokens of one text
    c = Cache(rng, "int8", 2, 64, 16, [256, 1, 1, 1])
    c.table[1:] = c.table[0]
    c.device()
    for shared in (128, 192, 256, 2 ** 31 - 1):
        check(c, [1, 1, 1, 1], [100, 130, 190, 256], 2, "f16", [0, 4], [shared])
        check(c, [3, 9, 1, 2], [100, 130, 190, 256], 2, "f32", [0, 4], [shared], window=70, sinks=3)


def test_groups_of_any_kind():
    """Groups that do not start at the first request, are empty, reach past the last; groups of
    requests of which one or none has tokens."""
    rng = np.random.default_rng(22)
    lengths = [150, 160, 170, 180, 190, 200]
    c = shared_cache(rng, "fp8", 2, 64, 16, [0, 6], lengths, [150])
    for groups, new in (([2, 4], [1] * 6), ([0, 0, 6, 6], [1] * 6), ([-3, 2, 99], [1] * 6),
                        ([3, 3, 3], [1] * 6), ([0, 3, 6], [0, 1, 0, 1, 2, 0]), ([0, 6], [0] * 5 + [1]),
                        ([0, 2, 4, 6], [0, 0, 1, 1, 0, 0])):
        check(c, new, lengths, 3, "f16", groups, [128] * (len(groups) - 1))


@pytest.mark.parametrize("n", [5, 200])
def test_the_first_requests_of_a_group_may_be_short(n):
    """Requests that ended, or have not reached the end of what the others share: their rows name
    none of the shared pages."""
    rng = np.random.default_rng(n)
    lengths = np.array([0, 3, 200, 210, 190] + [195] * (n - 5))
    c = Cache(rng, "fp8", 2, 64, 16, lengths)
    c.table[3:, :11] = c.table[2, :11]
    c.table[0] = -1
    c.device()
    for first, new in ((0, 0), (0, 1), (1, 2)):
        take = np.ones(n, int)
        take[:2] = 0, new
        check(c, take, lengths, 3, "f16", [first, n], [176])
        check(c, take, lengths, 1, "f32", [first, n], [176], window=60, sinks=20)


def test_rows_that_see_nothing():
    rng = np.random.default_rng(1)
    lengths, new = [140, 0, 150, 3], [2, 3, 1, 7]
    c = shared_cache(rng, "fp8", 2, 64, 16, [0, 4], [140, 140, 150, 140], [128])
    O = check(c, new, lengths, 2, "f16", [0, 4], [128])
    assert (O[2:5] == 0).all() and (O[6:10] == 0).all() and (O[10:] != 0).any()
    c.table[:, :] = -1
    c.device()
    assert (check(c, new, lengths, 2, "f32", [0, 4], [128]) == 0).all()


def test_missing_pages_and_short_tables():
    rng = np.random.default_rng(4)
    lengths = [300, 280, 290, 260]
    c = shared_cache(rng, "int8", 2, 128, 16, [0, 4], lengths, [256])
    c.table[:, 2:9] = -1                       # pages of the shared tokens that are gone
    c.table[2, 17] = c.k.shape[0]
    c.device()
    for new in ([1, 1, 1, 1], [4, 1, 9, 3]):
        check(c, new, lengths, 2, "f16", [0, 4], [256])
        check(c, new, lengths, 2, "f32", [0, 4], [256], window=140, sinks=4)
    c = shared_cache(rng, "fp8", 1, 64, 16, [0, 3], [400, 300, 350], [208], cols=13)
    for shared in (208, 300):
        check(c, [1, 3, 2], [400, 300, 350], 4, "f16", [0, 3], [shared])


def test_rows_of_no_request():
    rng = np.random.default_rng(6)
    c = shared_cache(rng, "fp8", 2, 64, 32, [0, 3], [150, 160, 170], [128])
    check(c, [1, 1, 1], [150, 160, 170], 2, "f16", [0, 3], [128], starts=[2, 3, 3, 6], n_tok=9)
    check(c, [1, 1, 1], [150, 160, 170], 2, "f16", [0, 3], [128], starts=[-4, 1, 3, 5], n_tok=20)
    check(c, [1, 1, 1], [150, 160, 170], 2, "f16", [0, 3], [128], starts=[0, 1, 30, 31], n_tok=20)


@pytest.mark.parametrize("out", ["f16", "f32"])
def test_uneven_scales(out):
    rng = np.random.default_rng(8)
    lengths = [200, 333, 194]
    c = Cache(rng, "int8", 2, 64, 16, lengths, spread=True)
    for r in (1, 2):
        c.table[r, :12] = c.table[0, :12]
    c.ks[c.table[0, 3]], c.vs[c.table[0, 4]], c.vs[c.table[1, 12]] = 0.0, 0.0, 0.0
    c.ks *= np.float32(1e-3)
    c.device()
    check(c, [1, 1, 1], lengths, 3, out, [0, 3], [192])
    check(c, [6, 2, 4], lengths, 3, out, [0, 3], [192])
    check(c, [1, 1, 1], lengths, 1, out, [0, 3], [192], scale=30.0)
    c.vs[:] = 0.0
    c.device()
    assert (check(c, [1, 9, 1], lengths, 1, out, [0, 3], [192]) == 0).all()


def test_many_requests_and_groups():
    """More than one workgroup's threads plan."""
    rng = np.random.default_rng(9)
    cuts = np.sort(rng.integers(0, 1201, 399))
    groups = np.concatenate([[0], cuts, [1200]])
    prefix = rng.integers(0, 200, 400)
    lengths = np.zeros(1200, int)
    for g in range(400):
        n = groups[g + 1] - groups[g]
        lengths[groups[g]:groups[g + 1]] = prefix[g] + rng.integers(0, 40, n)
    c = shared_cache(rng, "fp8", 1, 64, 16, groups, lengths, prefix)
    shared = prefix // 16 * 16
    check(c, (lengths > 0).astype(int), lengths, 2, "f16", groups, shared)
    check(c, np.minimum(lengths, rng.integers(0, 4, 1200)), lengths, 8, "f16", groups, shared)


@pytest.mark.parametrize("n,new", [(128, 1), (129, 1), (85, 3), (86, 3), (512, 1), (513, 1),
                                   (1024, 1), (1025, 1)])
def test_batches_at_the_sizes_where_the_plan_changes(n, new):
    """Each workgroup's own plan and one for all of them, from what is in LDS and from memory."""
    rng = np.random.default_rng(n)
    groups = np.concatenate([[0], np.sort(rng.integers(0, n + 1, n // 5)), [n]])
    prefix = rng.integers(0, 150, len(groups) - 1)
    lengths = np.zeros(n, int)
    for g, (r0, r1) in enumerate(zip(groups, groups[1:])):
        lengths[r0:r1] = prefix[g] + rng.integers(new, 20, r1 - r0)
    c = shared_cache(rng, "int8", 2, 64, 16, groups, lengths, prefix)
    check(c, [new] * n, lengths, 4, "f16", groups, prefix // 16 * 16)
    check(c, rng.integers(0, new + 1, n), lengths, 1, "f32", groups, prefix // 16 * 16, window=70, sinks=2)


@pytest.mark.parametrize("group,new", [(8, 3), (5, 5), (8, 4), (11, 3), (32, 2), (1, 96), (1, 97), (32, 3)])
def test_rows_of_a_request(group, new):
    """24, 25, 32, 33, 64, 96 and 97 rows a request, where sharing pays and where it does not."""
    rng = np.random.default_rng(group)
    lengths = [330, 300, 390, 301, 420]
    for groups, shared in (([0, 5], [192]), ([0, 2, 5], [128, 192])):
        c = shared_cache(rng, "fp8", 2, 64, 32, groups, lengths, shared)
        check(c, [new] * 5, lengths, group, "f16", groups, shared)
        check(c, [new, 1, 2 * new, 0, new], lengths, group, "f32", groups, shared, window=150, sinks=3)


def test_long_prefix_and_long_tails():
    rng = np.random.default_rng(10)
    lengths = [9000, 6100, 6050, 6047, 40, 7000]
    c = shared_cache(rng, "int8", 2, 64, 64, [0, 4, 6], lengths, [6047, 40])
    check(c, [1] * 6, lengths, 2, "f16", [0, 4, 6], [6016, 0])
    check(c, [2, 1, 0, 1, 1, 9], lengths, 9, "f32", [0, 4, 6], [6016, 0], window=3000, sinks=4)


def test_prompts_are_answered_too():
    """Requests of many rows each: nothing is gained by sharing, and the result is the same."""
    rng = np.random.default_rng(14)
    lengths = [300, 330, 310]
    c = shared_cache(rng, "fp8", 2, 64, 32, [0, 3], lengths, [192])
    check(c, [90, 100, 110], lengths, 2, "f16", [0, 3], [192])
    check(c, [33, 33, 33], lengths, 1, "f32", [0, 3], [192])
    check(c, [32, 32, 32], lengths, 1, "f32", [0, 3], [192])
    q = torch.randn(300, 256, device=DEV).half()
    args = c.kv, q, ints([0, 90, 190, 300]), ints(lengths), c.tab
    none = ints([])
    assert torch.equal(B.kv8_prefix_attention(*args, ints([0]), none, 4), B.kv8_attention(*args, 4))


@pytest.mark.parametrize("new,group", [([1] * 5, 1), ([2, 1, 3, 1, 1], 5), ([1] * 5, 16)])
def test_bad_codes_and_scales_stay_with_the_rows_that_see_them(new, group):
    """NaN codes and scales among shared and own keys, at places that only some rows see."""
    lengths = [200, 230, 260, 195, 210]
    for window in (0, 40, 120):
        c = shared_cache(np.random.default_rng(30), "fp8", 2, 64, 16, [0, 5], lengths, [192])
        c.v[c.table[0, 6], 0, 5, 3] = 0x7F              # a shared key: one dimension of its rows
        c.v[c.table[1, 13], 1, 9, 2] = 0xFF             # one of request 1's own
        c.ks[c.table[0, 2], 1] = np.nan                 # all of a page's rows, one head
        c.vs[c.table[2, 15], 0] = np.inf
        c.device()
        say(f"case: prefix, bad values, new={new} group={group} window={window}")
        rng = np.random.default_rng(3)
        Q = (2 * rng.standard_normal((sum(new), 2 * group * 64))).astype(np.float16)
        got = B.kv8_prefix_attention(
            c.kv, torch.from_numpy(Q).to(DEV), ints(np.concatenate([[0], np.cumsum(new)])),
            ints(lengths), c.tab, ints([0, 5]), ints([192]), 2 * group, window=window,
            odtype=torch.float32).double().cpu().numpy().reshape(sum(new), 2 * group, 64)
        ref, bound = row_reference(c, Q.astype(np.float64), new, lengths, group, window, 0, "f32")
        nan = np.isnan(ref)
        assert (np.isnan(got) == nan).all() and nan.any() and not nan.all()
        assert (np.where(nan, -1.0, np.abs(got - ref) - bound) <= 0).all()


def test_one_workspace_for_every_smaller_batch():
    rng = np.random.default_rng(15)
    lengths = [300] * 12
    c = shared_cache(rng, "int8", 2, 64, 32, [0, 12], lengths, [256])
    for H, n_tok in ((6, 700), (34, 40)):
        ws = B.kv8_prefix_attention_workspace(c.kv, 12, n_tok, H, DEV)
        ws[65536:] = 0xFF
        for r0, r1, new, groups in ((0, 12, 1, [0, 12]), (0, 1, 30, [0, 1]), (0, 12, 3, [0, 5, 12]),
                                    (3, 5, 1, [0, 2]), (0, 12, 2, list(range(13))), (2, 9, 1, [0, 7]),
                                    (0, 2, 10, [0, 2])):
            n = [new] * (r1 - r0)
            if sum(n) > n_tok:
                continue
            sub = Cache.__new__(Cache)
            sub.__dict__.update(c.__dict__, table=c.table[r0:r1], tab=c.tab[r0:r1])
            check(sub, n, lengths[r0:r1], H // 2, "f16", groups, [256] * (len(groups) - 1), ws=ws)


def test_pages_past_32_bits():
    """A cache of more than 4 GiB whose pages lie at its end: the same as in a small one."""
    say("case: prefix over 4 GiB")
    rng = np.random.default_rng(31)
    lengths = [700, 650, 660]
    c = shared_cache(rng, "int8", 8, 128, 128, [0, 3], lengths, [640])
    n, far = c.kv.k.shape[0], 33000
    kv = B.DeviceKV8.empty(far, 8, 128, 128, "int8", DEV)
    assert kv.k[:far - n].numel() > 2 ** 32
    for big, small in zip((kv.k, kv.v, kv.kscale, kv.vscale), (c.kv.k, c.kv.v, c.kv.kscale, c.kv.vscale)):
        big[far - n:] = small
    table = torch.where(c.tab >= 0, c.tab + (far - n), -1)
    q = torch.randn(3, 16 * 128, device=DEV).half()
    for new in ([1, 1, 1], [1, 2, 0]):
        args = (ints(np.concatenate([[0], np.cumsum(new)])), ints(lengths))
        for groups, shared in (([0, 3], [640]), ([0], [])):
            a = B.kv8_prefix_attention(c.kv, q, *args, c.tab, ints(groups), ints(shared), 16)
            b = B.kv8_prefix_attention(kv, q, *args, table, ints(groups), ints(shared), 16)
            assert torch.equal(a, b)
