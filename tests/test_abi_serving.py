"""Host checks of the serving calls (adapters, 8-bit cache, attention): every bad argument is
refused before any HIP call.  Nothing here reaches a GPU: each call fails validation or is a no-op,
and the pointers are placeholders that are never dereferenced."""
import ctypes as C
import os

import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import test_sanitize as S

OK, INVALID, UNSUPPORTED, RANGE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x10000  # 16-byte aligned placeholder address


def _adapters(n=4, r_max=16, d_in=256, d_out=64, A=P, lda=256, stride_a=4096, Bp=P, ldb=16,
              stride_b=1024, rank=P, scale=P):
    return B.Adapters(n, r_max, d_in, d_out, A, lda, stride_a, Bp, ldb, stride_b, rank, scale)


def _adapter(ad=None, X=P, xdt=B.DFS_F16, T=3, ldx=256, ids=P, base=P, ldbase=64, Y=P + 64,
             ydt=B.DFS_F16, ldy=64, ws=P, ws_bytes=0):
    """Every default but ws_bytes is fine; T = 300 needs a workspace."""
    ad = ad or _adapters()
    return B.lib().dict_adapter_forward(X, xdt, T, ldx, C.byref(ad), ids, base, ldbase, Y, ydt, ldy,
                                        ws, ws_bytes, None)


def test_adapter_validation():
    assert _adapter(T=0) == OK
    assert _adapter(T=0, ids=None, X=None, Y=None) == OK
    # a batch that needs a workspace and has too little passes every other check
    assert _adapter(T=300) == WORKSPACE
    assert _adapter(T=300, ws=None, ws_bytes=1 << 30) == WORKSPACE
    assert _adapter(T=300, ws=P + 8, ws_bytes=1 << 30) == ALIGN
    assert _adapter(T=-1) == INVALID
    for name in ("n", "r_max", "d_in", "d_out"):
        assert _adapter(_adapters(**{name: 0})) == INVALID
    for name in ("A", "Bp", "rank", "scale"):
        assert _adapter(_adapters(**{name: None})) == INVALID
    assert _adapter(_adapters(r_max=257, ldb=264)) == RANGE
    assert _adapter(_adapters(r_max=256, ldb=256), T=300) == WORKSPACE
    assert _adapter(_adapters(n=16001)) == RANGE
    assert _adapter(_adapters(lda=248)) == INVALID
    assert _adapter(_adapters(ldb=8)) == INVALID
    assert _adapter(_adapters(stride_a=-8)) == INVALID
    assert _adapter(_adapters(stride_b=-8)) == INVALID
    assert _adapter(_adapters(A=P + 8)) == ALIGN
    assert _adapter(_adapters(Bp=P + 2)) == ALIGN
    assert _adapter(_adapters(lda=260)) == ALIGN
    assert _adapter(_adapters(ldb=20)) == ALIGN
    assert _adapter(_adapters(stride_a=4100)) == ALIGN
    assert _adapter(_adapters(stride_b=1028)) == ALIGN
    assert _adapter(_adapters(rank=P + 2)) == ALIGN
    assert _adapter(_adapters(scale=P + 1)) == ALIGN
    assert _adapter(xdt=B.DFS_F32) == UNSUPPORTED
    assert _adapter(xdt=B.DFS_NVFP4) == UNSUPPORTED
    assert _adapter(ydt=B.DFS_FP8) == UNSUPPORTED
    assert _adapter(X=None) == INVALID
    assert _adapter(X=P + 2) == ALIGN
    assert _adapter(ldx=248) == INVALID
    assert _adapter(ldx=260) == ALIGN
    assert _adapter(Y=None) == INVALID
    assert _adapter(Y=P + 1) == ALIGN
    assert _adapter(Y=P + 2, ydt=B.DFS_F32) == ALIGN
    assert _adapter(ldy=63) == INVALID
    assert _adapter(ldbase=63) == INVALID
    assert _adapter(base=P + 1) == ALIGN
    assert _adapter(base=P, Y=P, ldbase=72) == INVALID       # in place with another stride
    assert _adapter(base=None, ldbase=0, T=300) == WORKSPACE  # no base: its stride is not looked at
    assert _adapter(ids=None) == INVALID
    assert _adapter(ids=P + 2) == ALIGN
    assert B.lib().dict_adapter_forward(P, B.DFS_F16, 1, 256, None, P, None, 0, P, B.DFS_F16, 64,
                                        P, 0, None) == INVALID


def test_adapter_workspace_size():
    n = C.c_size_t(0)
    ad = _adapters()
    f = B.lib().dict_adapter_workspace_size
    assert f(1, C.byref(ad), None) == INVALID
    assert f(-1, C.byref(ad), C.byref(n)) == INVALID
    assert f(1, None, C.byref(n)) == INVALID
    assert f(0, C.byref(ad), C.byref(n)) == OK and n.value == 0
    sizes = []
    for T in (300, 8192, 8193, 100000):
        assert f(T, C.byref(ad), C.byref(n)) == OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0


def _kv(n_pages=8, heads=2, head_dim=128, page=64, dtype=B.DFS_FP8, k=P, v=P, ks=P, vs=P):
    return B.KV8(n_pages, heads, head_dim, page, dtype, 0, k, v, ks, vs)


def _append(kv=None, n_req=2, n_tok=3, start=P, cached=P, table=P, ldt=4, pages=4, K=P, ldk=256,
            V=P, ldv=256, dtype=B.DFS_F16):
    kv = kv or _kv()
    return B.lib().kv8_append(C.byref(kv), n_req, n_tok, start, cached, table, ldt, pages, K, ldk, V,
                              ldv, dtype, None)


def _attend(kv=None, n_req=2, n_tok=3, start=P, length=P, table=P, ldt=4, pages=4, Q=P, ldq=512,
            q_heads=4, scale=0.1, window=0, sinks=0, O=P, odt=B.DFS_F16, ldo=512, ws=P, ws_bytes=16):
    """Every default but ws_bytes is fine."""
    kv = kv or _kv()
    return B.lib().kv8_attention(C.byref(kv), n_req, n_tok, start, length, table, ldt, pages, Q, ldq,
                                 q_heads, scale, window, sinks, O, odt, ldo, ws, ws_bytes, None)


BAD_CACHES = [(dict(n_pages=0), INVALID), (dict(heads=0), INVALID), (dict(heads=4097), RANGE),
              (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
              (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
              (dict(page=256), UNSUPPORTED), (dict(dtype=B.DFS_F16), UNSUPPORTED),
              (dict(dtype=B.DFS_NVFP4), UNSUPPORTED), (dict(k=None), INVALID),
              (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
              (dict(k=P + 8), ALIGN), (dict(v=P + 1), ALIGN), (dict(ks=P + 2), ALIGN),
              (dict(vs=P + 2), ALIGN)]
BAD_BATCHES = [(dict(n_req=-1), INVALID), (dict(n_tok=-1), INVALID), (dict(n_req=65536), RANGE),
               (dict(start=None), INVALID), (dict(table=None), INVALID), (dict(pages=0), INVALID),
               (dict(ldt=3), INVALID), (dict(pages=1 << 25, ldt=1 << 25), RANGE),
               (dict(start=P + 2), ALIGN), (dict(table=P + 1), ALIGN)]


@pytest.mark.parametrize("call", [_append, _attend])
def test_cache_and_batch_validation(call):
    for change, status in BAD_CACHES:
        assert call(kv=_kv(**change)) == status, change
    for change, status in BAD_BATCHES:
        assert call(**change) == status, change
    assert call(n_req=0) == OK and call(n_tok=0) == OK      # nothing to do


def test_append_validation():
    assert _append(cached=None) == INVALID
    assert _append(cached=P + 2) == ALIGN
    assert _append(K=None) == INVALID and _append(V=None) == INVALID
    assert _append(ldk=255) == INVALID and _append(ldv=255) == INVALID
    assert _append(K=P + 1) == ALIGN and _append(V=P + 2, dtype=B.DFS_F32) == ALIGN
    assert _append(dtype=B.DFS_FP8) == UNSUPPORTED


def test_attention_validation():
    assert _attend() == WORKSPACE                            # every other check passes
    assert _attend(ws=None, ws_bytes=1 << 40) == WORKSPACE
    assert _attend(ws=P + 4, ws_bytes=1 << 40) == ALIGN
    for dim in (64, 96, 128, 256):
        assert _attend(kv=_kv(head_dim=dim), ldq=4 * dim, ldo=4 * dim) == WORKSPACE
    assert _attend(length=None) == INVALID
    assert _attend(q_heads=0) == INVALID and _attend(q_heads=3) == INVALID
    assert _attend(kv=_kv(heads=2), q_heads=4098) == RANGE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(scale=scale) == INVALID
    assert _attend(sinks=-1) == INVALID
    assert _attend(window=-1) == WORKSPACE                   # no window
    assert _attend(Q=None) == INVALID and _attend(O=None) == INVALID
    assert _attend(ldq=504) == INVALID and _attend(ldo=511) == INVALID
    assert _attend(ldq=516) == ALIGN
    assert _attend(Q=P + 8) == ALIGN
    assert _attend(O=P + 1) == ALIGN and _attend(O=P + 2, odt=B.DFS_F32) == ALIGN
    assert _attend(O=P + 2) == WORKSPACE                     # f16 O at any element
    assert _attend(odt=B.DFS_INT8) == UNSUPPORTED


def test_attention_workspace_size():
    n = C.c_size_t(0)
    kv = _kv()
    f = B.lib().kv8_attention_workspace_size
    assert f(C.byref(kv), 1, 1, 4, None) == INVALID
    assert f(C.byref(kv), -1, 1, 4, C.byref(n)) == INVALID
    assert f(C.byref(kv), 1, 1, 3, C.byref(n)) == INVALID
    assert f(C.byref(kv), 65536, 1, 4, C.byref(n)) == RANGE
    assert f(C.byref(_kv(page=17)), 1, 1, 4, C.byref(n)) == UNSUPPORTED
    assert f(C.byref(kv), 0, 0, 4, C.byref(n)) == OK and n.value >= 65536
    assert f(C.byref(kv), 3, 100000, 4, C.byref(n)) == OK and n.value >= 65536


def test_binding_checks():
    z = lambda dt, *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    h, f, i = torch.float16, torch.float32, torch.int32
    A, Bm, rank, scale = z(h, 3, 8, 64), z(h, 3, 40, 8), z(i, 3), z(f, 3)
    ad = B.DeviceAdapters(A, Bm, rank, scale)
    assert (ad.r_max, ad.d_in, ad.d_out) == (8, 64, 40)
    for bad in ((A[:2], Bm, rank, scale), (A, Bm[:, :, ::2], rank, scale), (A, Bm, z(i, 2), scale),
                (A, Bm, z(torch.int64, 3), scale), (A, Bm, rank, z(h, 3)), (A[:, :7], Bm, rank,
                                                                            scale),
                (z(h, 3, 8, 60), Bm, rank, scale)):          # last row ends inside a piece of 8
        with pytest.raises(ValueError):
            B.DeviceAdapters(*bad)
    with pytest.raises(TypeError):
        B.DeviceAdapters(A.float(), Bm, rank, scale)
    X, ids = z(h, 5, 64), z(i, 5)
    for kw in (dict(X=X[:, :56]), dict(ids=z(i, 4)), dict(ids=z(torch.int64, 5)),
               dict(Y=z(h, 4, 40)), dict(base=z(h, 5, 39)), dict(X=z(h, 64, 5).t())):
        with pytest.raises(ValueError):
            B.dict_adapter_forward(**{"X": X, "ad": ad, "ids": ids, **kw})
    with pytest.raises(TypeError):
        B.dict_adapter_forward(X, ad, ids, base=z(f, 5, 40))
    with pytest.raises(TypeError):
        B.dict_adapter_forward(X.bfloat16(), ad, ids)

    kv = B.DeviceKV8.empty(4, 2, 64, 16, "int8", "cpu")
    u8 = torch.uint8
    with pytest.raises(ValueError):
        B.DeviceKV8.empty(4, 2, 64, 16, "int4", "cpu")
    with pytest.raises(ValueError):
        B.DeviceKV8(kv.k, z(u8, 4, 2, 16, 64), kv.kscale, kv.vscale, "fp8")   # values: dims first
    with pytest.raises(ValueError):
        B.DeviceKV8(kv.k, kv.v, kv.kscale[:, :1], kv.vscale, "fp8")
    with pytest.raises(ValueError):
        B.DeviceKV8(kv.k.transpose(2, 3), kv.v, kv.kscale, kv.vscale, "fp8")
    K, start, have, table = z(h, 3, 128), z(i, 3), z(i, 2), z(i, 2, 4)
    good = dict(kv=kv, K=K, V=K, tok_start=start, cached=have, table=table)
    for kw in (dict(K=K[:, :64]), dict(V=K[:2]), dict(tok_start=have), dict(table=table[:1]),
               dict(table=table.long()), dict(cached=z(torch.int64, 2)), dict(table=table.t())):
        with pytest.raises(ValueError):
            B.kv8_append(**{**good, **kw})
    with pytest.raises(TypeError):
        B.kv8_append(**{**good, "V": K.float()})
    good = dict(kv=kv, Q=z(h, 3, 256), tok_start=start, length=have, table=table, q_heads=4)
    for kw in (dict(Q=z(h, 3, 128)), dict(O=z(h, 2, 256)), dict(q_heads=8), dict(length=z(i, 3))):
        with pytest.raises(ValueError):
            B.kv8_attention(**{**good, **kw})
    with pytest.raises(TypeError):
        B.kv8_attention(**{**good, "Q": z(f, 3, 256)})


def test_host_code_under_clang_asan_ubsan():
    """These checks against the copy of the library whose host code is sanitized."""
    import glob

    from dictionary_factored_sparse_amd import build as hb
    if os.environ.get("DFS_LIB_PATH"):
        pytest.skip("this is that run")
    rt = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not rt:
        pytest.skip("clang's ASan runtime is not installed")
    lib = hb.build_host_sanitized()
    out = S._run({"DFS_LIB_PATH": lib, "LD_PRELOAD": rt[-1]}, ["tests/test_abi_serving.py"])
    assert " passed" in out
