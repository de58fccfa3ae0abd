"""The Python binding of the serving calls, on the CPU: what it allocates and where, and what it
refuses before the library sees a pointer."""
import contextlib

import pytest
import torch

from dictionary_factored_sparse_amd import binding as B

z = lambda dt, *s: torch.zeros(*s, dtype=dt)  # noqa: E731
h, f, i = torch.float16, torch.float32, torch.int32


class Streams:
    """Stands for torch.cuda's streams: which one is current, and on which tensors were made."""

    class Stream:
        device = torch.device("cpu")

        def __init__(self, n):
            self.cuda_stream = n

    def __init__(self, patch):
        self.side, self.now, self.made, self.launched = self.Stream(7), self.Stream(1), [], []
        patch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        patch.setattr(torch.cuda, "stream", self.use)
        patch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
        patch.setattr(B, "_on_device", lambda *a: None, raising=False)
        patch.setattr(B, "_stream_of", lambda t, *given: (
            given[0] if given and given[0] is not None else self.now).cuda_stream)
        for name in ("empty", "zeros"):
            make = getattr(torch, name)
            patch.setattr(torch, name, lambda *a, make=make, **k: (
                self.made.append(self.now.cuda_stream), make(*a, **k))[1])
        patch.setattr(B, "lib", lambda: self)

    @contextlib.contextmanager
    def use(self, s):
        was, self.now = self.now, s
        yield
        self.now = was

    def __getattr__(self, name):      # the library
        def call(*args):
            if name.endswith("workspace_size"):
                args[-1]._obj.value = 70000
            elif name == "dict_csc_capacity":
                return 16
            else:
                self.launched.append(args[-1])
            return 0
        return call


def serving_calls():
    ad = B.DeviceAdapters(z(h, 3, 8, 64), z(h, 3, 40, 8), z(i, 3), z(f, 3))
    kv = B.DeviceKV8.empty(4, 2, 64, 16, "int8", "cpu")
    K, start, have, table = z(h, 3, 128), z(i, 3), z(i, 2), z(i, 2, 4)
    return [(B.dict_adapter_forward, (K[:, :64], ad, z(i, 3))),
            (B.kv8_append, (kv, K, K, start, have, table)),
            (B.kv8_attention, (kv, z(h, 3, 256), start, have, table, 4))]


def test_what_a_call_makes_is_made_on_its_stream(monkeypatch):
    calls = serving_calls()
    s = Streams(monkeypatch)
    for fn, args in calls:
        for stream in (None, s.side, s.now):
            s.made.clear()
            s.launched.clear()
            fn(*args, stream=stream)
            want = (stream or s.now).cuda_stream
            assert s.launched == [want] and set(s.made) <= {want}, (fn.__name__, stream)
            assert s.made or fn is B.kv8_append
            assert s.now.cuda_stream == 1


def test_the_projections_calls_too(monkeypatch):
    """The same of the calls that pack, multiply and prune."""
    D = B.DeviceDict.from_atoms(z(h, 16, 64))
    c = B.DeviceCSC(16, 40, 8, z(i, 41), z(torch.int16, 16), vals=z(h, 16))
    q = B.DeviceNVFP4.empty(32, "cpu")
    X, Z, W, S = z(h, 3, 64), z(f, 3, 16), z(f, 16, 40), z(f, 64, 64)
    calls = [(B.dict_group_forward, ([X], D, [c])), (B.dict_multi_forward, ([X], [D], [c])),
             (B.dict_proj_forward, (X, D, c)), (B.dict_xd_forward, ([X], D)),
             (B.dict_zc_forward, (Z, 3, [c])), (B.nvfp4_pack, (W,)), (B.nvfp4_unpack, (q,)),
             (B.dict_pack_csc, (z(h, 16, 40),)), (B.dict_pack_bcsc, (z(h, 16, 40),)),
             (B.csc_quantize8, (c, "fp8")), (B.csc_to_nvfp4, (c,)),
             (B.dict_gram_inverse, (D, S, 0.1)), (B.dict_obs_prune, (W, z(f, 16, 16), 4)),
             (B.dict_refit, (z(f, 64, 40), W, 0.1))]
    s = Streams(monkeypatch)
    for fn, args in calls:
        for stream in (None, s.side, s.now):
            s.made.clear()
            s.launched.clear()
            fn(*args, stream=stream)
            want = (stream or s.now).cuda_stream
            assert set(s.launched) == {want} and set(s.made) == {want}, (fn.__name__, stream)
            assert s.now.cuda_stream == 1
    s.launched.clear()
    B.nvfp4_pack(W, s.side)                                  # by position
    assert s.launched == [7]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    calls = serving_calls() + [(B.nvfp4_pack, (z(f, 16, 40),))]
    s = Streams(monkeypatch)
    s.side.device = torch.device("meta")
    for fn, args in calls:
        with pytest.raises(ValueError, match="stream of"):
            fn(*args, stream=s.side)
    assert not s.launched


class Refusing:
    """A library that must not be reached: the addresses would be the host's."""

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *args: 0
        raise AssertionError(f"{name} was called")


def test_tensors_of_the_host_are_refused(monkeypatch):
    calls = serving_calls()
    monkeypatch.setattr(B, "lib", lambda: Refusing())
    for fn, args in calls:
        with pytest.raises(ValueError, match="GPU"):
            fn(*args)


def test_a_workspace_is_on_the_inputs_device_and_counted_in_bytes(monkeypatch):
    calls = serving_calls()
    s = Streams(monkeypatch)
    got = []
    monkeypatch.setattr(Streams, "__getattr__",
                        lambda self, name: lambda *args: got.append(args[-2]) or 0)
    for fn, args in (calls[0], calls[2]):
        fn(*args, ws=z(i, 1000))
        fn(*args, ws=z(torch.uint8, 1000))
        for bad in (torch.empty(1000, dtype=torch.uint8, device="meta"), z(torch.uint8, 2000)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                fn(*args, ws=bad)
    assert got == [4000, 1000] * 2


def test_adapter_workspace_holds_every_smaller_batch():
    """The size rises with T, and no call of up to T tokens asks for more: the library is given
    the size for T and reaches its next check (a workspace that is not aligned) at every T'."""
    import ctypes as C
    P, n = 0x10000, C.c_size_t(0)
    lib = B.lib()
    steps = sorted({*range(1, 600), *range(600, 9000, 7), 1151, 1152, 4099, 7679, 7680, 8191, 8192,
                    8193, 8194, 12000, 16384, 40000, 100000, 1000003})
    for pool, r, d_in, d_out in ((24, 64, 11008, 4096), (8, 32, 4096, 4096), (1, 8, 64, 64),
                                 (1, 256, 5120, 96), (512, 16, 2048, 2048), (5000, 64, 8192, 256),
                                 (16000, 33, 1000, 500), (3, 200, 30000, 64)):
        ad = B.Adapters(pool, r, d_in, d_out, P, -(-d_in // 8) * 8, 0, P, -(-r // 8) * 8, 0, P, P)

        def forward(T, size):
            return lib.dict_adapter_forward(P, B.DFS_F16, T, -(-d_in // 8) * 8, C.byref(ad), P,
                                            None, 0, P, B.DFS_F16, d_out, P + 8, size, None)

        sizes = []
        for T in steps:
            assert lib.dict_adapter_workspace_size(T, C.byref(ad), C.byref(n)) == 0
            sizes.append(n.value)
        assert sizes == sorted(sizes), (pool, r, d_in)
        for T, size in zip(steps, sizes):
            if size:                # 4: past the check of the size; none needed reaches no launch
                assert forward(T, size) == 4, (pool, r, d_in, T)


def test_attention_workspace_holds_every_smaller_batch():
    """The size rises with the requests and with the tokens, and no call of up to that many asks
    for more (as above: the check after the size's is reached)."""
    import ctypes as C
    P, n = 0x10000, C.c_size_t(0)
    lib = B.lib()
    reqs = [1, 2, 3, 5, 15, 16, 17, 32, 33, 63, 255, 256, 257, 1000, 65535]
    toks = [1, 2, 4, 8, 15, 16, 17, 31, 32, 33, 64, 100, 512, 1000, 4097, 8192, 70000]
    for heads, group, dim in ((8, 1, 128), (8, 4, 128), (4, 3, 64), (2, 17, 96), (1, 32, 256)):
        kv = B.KV8(8, heads, dim, 64, B.DFS_FP8, 0, P, P, P, P)
        H, size = heads * group, {}
        for r in reqs:
            for t in toks:
                assert lib.kv8_attention_workspace_size(C.byref(kv), r, t, H, C.byref(n)) == 0
                size[r, t] = n.value
                assert lib.kv8_attention(C.byref(kv), r, t, P, P, P, 4, 4, P, H * dim, H, 0.1, 0, 0,
                                         P, B.DFS_F16, H * dim, P + 8, n.value, None) == 4
        for a, b in zip(reqs, reqs[1:]):
            assert all(size[a, t] <= size[b, t] for t in toks), (heads, group, dim, a)
        for a, b in zip(toks, toks[1:]):
            assert all(size[r, a] <= size[r, b] for r in reqs), (heads, group, dim, a)
