"""Host checks of the calls for pages, beams and shared prefixes: every bad argument is refused
before any HIP call.  Nothing here reaches a GPU: each call fails validation or is a no-op, and the
pointers are placeholders that are never dereferenced."""
import ctypes as C

import pytest

from dictionary_factored_sparse_amd import binding as B
from tests.test_abi_serving import BAD_BATCHES, BAD_CACHES, _kv

OK, INVALID, UNSUPPORTED, RANGE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x10000  # 16-byte aligned placeholder address
BAD_POOLS = [(dict(n_pages=0), INVALID), (dict(n_pages=(1 << 28) + 1), RANGE),
             (dict(refs=None), INVALID), (dict(refs=P + 2), ALIGN)]
BAD_PAGES = [(dict(page=0), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED)]


def _tables(n_req=2, page=64, n_pages=8, refs=P, cached=P, new=P, n_tok=3, table=P, ldt=4, pages=4,
            start=5 * P, length=2 * P, req=P, pos=P, slot=P, missing=None):
    """Every default but missing is fine."""
    return B.lib().kv8_tables(n_req, page, n_pages, refs, cached, new, n_tok, table, ldt, pages,
                              start, length, req, pos, slot, missing, None)


def test_tables_validation():
    assert _tables() == INVALID                    # every other check passes: see missing below
    for change, status in BAD_POOLS + BAD_PAGES:
        assert _tables(missing=6 * P, **change) == status, change
    for change, status in ((dict(n_req=-1), INVALID), (dict(n_req=65536), RANGE),
                           (dict(n_tok=-1), INVALID), (dict(pages=0), INVALID),
                           (dict(ldt=3), INVALID), (dict(pages=1 << 25, ldt=1 << 25), RANGE),
                           (dict(table=None), INVALID), (dict(table=P + 1), ALIGN),
                           (dict(cached=None), INVALID), (dict(new=None), INVALID),
                           (dict(start=None), INVALID), (dict(length=None), INVALID),
                           (dict(cached=P + 1), ALIGN), (dict(new=P + 2), ALIGN),
                           (dict(start=P + 2), ALIGN), (dict(length=P + 3), ALIGN),
                           (dict(req=P + 2), ALIGN), (dict(pos=P + 2), ALIGN),
                           (dict(slot=P + 4), ALIGN), (dict(missing=P + 2), ALIGN)):
        assert _tables(**{"missing": 6 * P, **change}) == status, change
    for out, n in (("length", 2), ("start", 3), ("missing", 1)):      # over cached or n_new
        for at in (P - 4 * (n - 1), P, P + 4):
            assert _tables(**{"missing": 6 * P, "new": 3 * P, out: at}) == INVALID, (out, at)
            assert _tables(**{"missing": 6 * P, "cached": 3 * P, out: at}) == INVALID, (out, at)


def _release(n_req=2, n_pages=8, refs=P, table=P, ldt=4, pages=4, first=P, last=P):
    return B.lib().kv8_release(n_req, n_pages, refs, table, ldt, pages, first, last, None)


def test_release_validation():
    for change, status in BAD_POOLS:
        assert _release(**change) == status, change
    for change, status in ((dict(n_req=-1), INVALID), (dict(n_req=65536), RANGE),
                           (dict(pages=0), INVALID), (dict(ldt=3), INVALID),
                           (dict(pages=1 << 27, ldt=1 << 27), RANGE),
                           (dict(table=None), INVALID), (dict(table=P + 2), ALIGN),
                           (dict(first=P + 1), ALIGN), (dict(last=P + 2), ALIGN)):
        assert _release(**change) == status, change
    assert _release(n_req=0) == OK and _release(n_req=0, table=None) == OK


def _reorder(n_in=2, n_out=3, page=64, n_pages=8, refs=P, table=P, ldt=4, length=P, parent=P, keep=0,
             out=2 * P, ldo=4, pages=4, length_out=3 * P, src=4 * P, dst=5 * P, missing=P, ws=P, ws_bytes=15):
    """Every default but ws_bytes is fine."""
    return B.lib().kv8_reorder(n_in, n_out, page, n_pages, refs, table, ldt, length, parent, keep,
                               out, ldo, pages, length_out, src, dst, missing, ws, ws_bytes, None)


def test_reorder_validation():
    assert _reorder() == WORKSPACE                 # every other check passes
    assert _reorder(ws=None, ws_bytes=99) == WORKSPACE
    assert _reorder(ws=P + 8, ws_bytes=99) == ALIGN
    for change, status in BAD_POOLS + BAD_PAGES:
        assert _reorder(**change) == status, change
    for change, status in ((dict(n_in=-1), INVALID), (dict(n_out=-1), INVALID),
                           (dict(n_in=65536), RANGE), (dict(n_out=65536), RANGE),
                           (dict(pages=0), INVALID), (dict(ldt=3), INVALID), (dict(ldo=3), INVALID),
                           (dict(table=None), INVALID), (dict(out=None), INVALID),
                           (dict(length=None), INVALID), (dict(parent=None), INVALID),
                           (dict(length_out=None), INVALID), (dict(src=None), INVALID),
                           (dict(dst=None), INVALID), (dict(missing=None), INVALID),
                           (dict(table=P + 2), ALIGN), (dict(out=2 * P + 1), ALIGN),
                           (dict(length=P + 2), ALIGN), (dict(parent=P + 2), ALIGN),
                           (dict(length_out=P + 2), ALIGN), (dict(src=P + 2), ALIGN),
                           (dict(dst=P + 1), ALIGN), (dict(missing=P + 2), ALIGN)):
        assert _reorder(**change) == status, change
    for out in ("length_out", "src", "dst"):       # over what is read, and each other
        for at in (P, P + 4, P - 8):
            assert _reorder(**{"parent": 9 * P, out: at}) == INVALID, (out, at)
            assert _reorder(**{"length": 9 * P, out: at}) == INVALID, (out, at)
        assert _reorder(**{out: 8 * P}) == WORKSPACE
    assert _reorder(src=5 * P + 8) == INVALID and _reorder(dst=3 * P) == INVALID
    assert _reorder(src=3 * P - 8) == INVALID
    # rows that overlap: in place, and by one entry at either end
    assert _reorder(out=P) == INVALID
    assert _reorder(out=P + 4 * 7) == INVALID and _reorder(out=P + 4 * 8) == WORKSPACE
    assert _reorder(out=P - 4 * 11) == INVALID and _reorder(out=P - 4 * 12) == WORKSPACE


def test_reorder_workspace_size():
    n = C.c_size_t(0)
    f = B.lib().kv8_reorder_workspace_size
    assert f(1, None) == INVALID and f(-1, C.byref(n)) == INVALID and f(65536, C.byref(n)) == RANGE
    assert f(0, C.byref(n)) == OK and n.value == 0
    for rows in (1, 31, 32, 33, 65535):
        assert f(rows, C.byref(n)) == OK and n.value >= 8 * rows


def _copy(kvs, n=3, src=P, dst=P, length=P):
    a = (B.KV8 * max(len(kvs), 1))(*kvs)
    return B.lib().kv8_copy_pages(len(kvs), a, n, src, dst, length, None)


def test_copy_validation():
    for change, status in BAD_CACHES:
        assert _copy([_kv(), _kv(**change)]) == status, change
    for other in (dict(heads=3), dict(head_dim=64), dict(page=32), dict(n_pages=9)):
        assert _copy([_kv(), _kv(**other)]) == INVALID
    assert _copy([_kv()] * 17) == RANGE
    assert _copy([_kv()], n=-1) == INVALID
    assert _copy([_kv()], src=None) == INVALID and _copy([_kv()], dst=None) == INVALID
    assert _copy([_kv()], src=P + 2) == ALIGN and _copy([_kv()], dst=P + 1) == ALIGN
    assert _copy([_kv()], length=P + 2) == ALIGN
    assert _copy([], src=None) == OK and _copy([_kv()], n=0, src=None) == OK
    assert B.lib().kv8_copy_pages(1, None, 1, P, P, None, None) == INVALID
    assert B.lib().kv8_copy_pages(-1, None, 1, P, P, None, None) == INVALID


def _beam(n_req=2, width=4, vocab=100, logits=P, dt=B.DFS_F16, ldl=100, score=P, done=P, norm=P, eos=2,
          parent=2 * P, token=3 * P, score_out=4 * P, done_out=5 * P, ws=P, ws_bytes=16):
    """Every default but ws_bytes is fine."""
    return B.lib().beam_select(n_req, width, vocab, logits, dt, ldl, score, done, norm, eos, parent,
                               token, score_out, done_out, ws, ws_bytes, None)


def test_beam_validation():
    assert _beam() == WORKSPACE                    # every other check passes
    assert _beam(ws=None, ws_bytes=1 << 40) == WORKSPACE
    assert _beam(ws=P + 8, ws_bytes=1 << 40) == ALIGN
    for change, status in ((dict(n_req=-1), INVALID), (dict(width=0), INVALID),
                           (dict(vocab=0), INVALID), (dict(width=33), RANGE),
                           (dict(n_req=8193, width=1), RANGE), (dict(n_req=1025, width=8), RANGE),
                           (dict(vocab=(1 << 30) + 1, ldl=1 << 31), RANGE),
                           (dict(dt=B.DFS_FP8), UNSUPPORTED), (dict(dt=B.DFS_NVFP4), UNSUPPORTED),
                           (dict(ldl=99), INVALID), (dict(eos=-1), INVALID),
                           (dict(eos=100), INVALID), (dict(logits=None), INVALID),
                           (dict(score=None), INVALID), (dict(parent=None), INVALID),
                           (dict(token=None), INVALID), (dict(score_out=None), INVALID),
                           (dict(logits=P + 1), ALIGN), (dict(logits=P + 2, dt=B.DFS_F32), ALIGN),
                           (dict(score=P + 2), ALIGN), (dict(done=P + 2), ALIGN),
                           (dict(norm=P + 1), ALIGN), (dict(parent=P + 2), ALIGN),
                           (dict(token=P + 2), ALIGN), (dict(score_out=P + 2), ALIGN),
                           (dict(done_out=P + 2), ALIGN)):
        assert _beam(**change) == status, change
    for name in ("parent", "token", "score_out", "done_out"):
        assert _beam(**{name: P}) == INVALID and _beam(**{name: P + 28}) == INVALID
    for a, b in ((dict(token=2 * P + 28), dict(token=2 * P + 32)), (dict(score_out=2 * P), dict(score_out=6 * P)),
                 (dict(done_out=4 * P - 28), dict(done_out=4 * P - 32))):
        assert _beam(**a) == INVALID and _beam(**b) == WORKSPACE
    assert _beam(done=None, eos=-1) == WORKSPACE and _beam(done_out=None, norm=None) == WORKSPACE
    assert _beam(logits=P + 2) == WORKSPACE        # f16 logits at any element
    assert _beam(n_req=0, logits=None) == OK


def test_beam_workspace_holds_every_smaller_call():
    n = C.c_size_t(0)
    f = B.lib().beam_select_workspace_size
    assert f(1, 1, 1, None) == INVALID and f(-1, 1, 1, C.byref(n)) == INVALID
    assert f(1, 33, 1, C.byref(n)) == RANGE and f(0, 1, 1, C.byref(n)) == OK
    for req, width, vocab in ((1, 4, 32000), (24, 5, 50021), (8, 32, 131072), (64, 1, 700), (3, 2, 1)):
        assert f(req, width, vocab, C.byref(n)) == OK and n.value >= 65536
        for r in {1, 2, req // 2, req}:
            for w in {1, width // 2, width}:
                for v in {1, 7, 2048, 2049, 8193, vocab // 3, vocab - 1, vocab}:
                    for dt in (B.DFS_F16, B.DFS_F32):
                        if 1 <= r <= req and 1 <= w <= width and 1 <= v <= vocab:
                            # 4: past the check of the size, at one of the address
                            assert _beam(r, w, v, dt=dt, ldl=v, eos=0, ws=P + 8,
                                         ws_bytes=n.value) == ALIGN


def _prefix(kv=None, n_req=2, n_tok=3, start=P, length=P, table=P, ldt=4, pages=4, n_groups=1,
            groups=P, shared=P, Q=P, ldq=512, q_heads=4, scale=0.1, window=0, sinks=0, O=P,
            odt=B.DFS_F16, ldo=512, ws=P, ws_bytes=16):
    """Every default but ws_bytes is fine."""
    kv = kv or _kv()
    return B.lib().kv8_prefix_attention(C.byref(kv), n_req, n_tok, start, length, table, ldt, pages,
                                        n_groups, groups, shared, Q, ldq, q_heads, scale, window,
                                        sinks, O, odt, ldo, ws, ws_bytes, None)


def test_prefix_attention_validation():
    for change, status in BAD_CACHES:
        assert _prefix(kv=_kv(**change)) == status, change
    for change, status in BAD_BATCHES:
        assert _prefix(**{"n_groups": 0, **change}) == status, change
    assert _prefix() == WORKSPACE                  # every other check passes
    assert _prefix(ws=None, ws_bytes=1 << 40) == WORKSPACE
    assert _prefix(ws=P + 4, ws_bytes=1 << 40) == ALIGN
    for dim in (64, 96, 128, 256):
        assert _prefix(kv=_kv(head_dim=dim), ldq=4 * dim, ldo=4 * dim) == WORKSPACE
    assert _prefix(n_groups=-1) == INVALID and _prefix(n_groups=3) == INVALID
    assert _prefix(groups=None) == INVALID and _prefix(shared=None) == INVALID
    assert _prefix(groups=P + 2) == ALIGN and _prefix(shared=P + 1) == ALIGN
    assert _prefix(n_groups=0, groups=None, shared=None) == WORKSPACE
    assert _prefix(length=None) == INVALID
    assert _prefix(q_heads=0) == INVALID and _prefix(q_heads=3) == INVALID
    assert _prefix(kv=_kv(heads=2), q_heads=4098) == RANGE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _prefix(scale=scale) == INVALID
    assert _prefix(sinks=-1) == INVALID and _prefix(window=-1) == WORKSPACE
    assert _prefix(Q=None) == INVALID and _prefix(O=None) == INVALID
    assert _prefix(ldq=504) == INVALID and _prefix(ldo=511) == INVALID
    assert _prefix(ldq=516) == ALIGN and _prefix(Q=P + 8) == ALIGN
    assert _prefix(O=P + 1) == ALIGN and _prefix(O=P + 2, odt=B.DFS_F32) == ALIGN
    assert _prefix(odt=B.DFS_INT8) == UNSUPPORTED
    assert _prefix(n_req=0, n_groups=0) == OK and _prefix(n_tok=0) == OK


@pytest.mark.parametrize("dim,heads,group", [(64, 2, 1), (128, 8, 4), (256, 1, 40), (96, 3, 5)])
def test_prefix_workspace_holds_every_smaller_call(dim, heads, group):
    n = C.c_size_t(0)
    kv, H = _kv(heads=heads, head_dim=dim), heads * group
    f = B.lib().kv8_prefix_attention_workspace_size
    assert f(C.byref(kv), 1, 1, H, None) == INVALID and f(C.byref(kv), -1, 1, H, C.byref(n)) == INVALID
    assert f(C.byref(kv), 65536, 1, H, C.byref(n)) == RANGE
    for n_req, n_tok in ((1, 1), (4, 4), (64, 64), (7, 300), (200, 1000), (1500, 40)):
        assert f(C.byref(kv), n_req, n_tok, H, C.byref(n)) == OK and n.value >= 65536
        for r in {1, 2, 5, n_req // 3, n_req - 1, n_req}:
            for t in {1, 2, r, 2 * r, 16 * r // group, 16 * r // group + 1, 32 * r // group,
                      32 * r // group + 1, 33 * r, n_tok // 2, n_tok}:
                for g in {0, 1, 2, r // 2, r}:
                    if 1 <= r <= n_req and 1 <= t <= n_tok and 0 <= g <= r:
                        # 4: past the check of the size, at one of the address
                        assert _prefix(kv, r, t, n_groups=g, q_heads=H, ldq=H * dim, ldo=H * dim,
                                       ws=P + 4, ws_bytes=n.value) == ALIGN, (r, t, g)
