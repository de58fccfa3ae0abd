"""The Python binding of the calls for pages, beams and shared prefixes, on the CPU: what it
allocates and where, and what it refuses before the library sees a pointer."""
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests.test_serving_binding import Refusing, Streams, z

h, f, i, u8 = torch.float16, torch.float32, torch.int32, torch.uint8


def calls():
    kv = B.DeviceKV8.empty(4, 2, 64, 16, "int8", "cpu")
    refs, table, two, three = z(i, 9), z(i, 2, 4), z(i, 2), z(i, 3)
    return [(B.kv8_tables, (refs, 16, two, two, table, None, 5)),
            (B.kv8_release, (refs, table, two)),
            (B.kv8_reorder, (refs, 16, table, two, three, z(i, 3, 4))),
            (B.kv8_copy_pages, ([kv, kv], three, three, three)),
            (B.beam_select, (z(h, 6, 50), z(f, 6), 3, 1, z(i, 6), z(f, 6))),
            (B.kv8_prefix_attention, (kv, z(h, 3, 256), three, two, table, two, z(i, 1), 4))]


def test_what_a_call_makes_is_made_on_its_stream(monkeypatch):
    todo = calls()
    s = Streams(monkeypatch)
    for fn, args in todo:
        for stream in (None, s.side, s.now):
            s.made.clear()
            s.launched.clear()
            fn(*args, stream=stream)
            want = (stream or s.now).cuda_stream
            assert s.launched == [want] and set(s.made) <= {want}, (fn.__name__, stream)
            assert s.made or fn in (B.kv8_release, B.kv8_copy_pages)
            assert s.now.cuda_stream == 1


def test_a_stream_of_another_device_is_refused(monkeypatch):
    todo = calls()
    s = Streams(monkeypatch)
    s.side.device = torch.device("meta")
    for fn, args in todo:
        with pytest.raises(ValueError, match="stream of"):
            fn(*args, stream=s.side)
    assert not s.launched


def test_tensors_of_the_host_are_refused(monkeypatch):
    todo = calls()
    monkeypatch.setattr(B, "lib", lambda: Refusing())
    for fn, args in todo:
        with pytest.raises(ValueError, match="GPU"):
            fn(*args)


def test_one_tensor_elsewhere_is_refused(monkeypatch):
    """Each tensor of each call, on another device than the others."""
    monkeypatch.setattr(B, "lib", lambda: Refusing())
    monkeypatch.setattr(B, "_stream_of", lambda t: 0)
    monkeypatch.setattr(B, "_on_device", lambda ts, what: B._same_device(ts, what))
    for fn, args in calls():
        for k, a in enumerate(args):
            if isinstance(a, torch.Tensor):
                bad = list(args)
                bad[k] = torch.empty_like(a, device="meta")
                with pytest.raises((ValueError, AssertionError, RuntimeError)) as e:
                    fn(*bad)
                assert "was called" not in str(e.value), (fn.__name__, k)


def test_workspaces_are_on_the_inputs_device_and_counted_in_bytes(monkeypatch):
    todo = calls()
    Streams(monkeypatch)
    got = []
    monkeypatch.setattr(Streams, "__getattr__",
                        lambda self, name: lambda *args: got.append(args[-2]) or 0)
    for fn, args in (todo[2], todo[4], todo[5]):
        fn(*args, ws=z(i, 1000))
        fn(*args, ws=z(u8, 1000))
        for bad in (torch.empty(1000, dtype=u8, device="meta"), z(u8, 2000)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                fn(*args, ws=bad)
    assert got == [4000, 1000] * 3


def test_shapes_and_types_are_checked(monkeypatch):
    Streams(monkeypatch)
    refs, table, two, three = z(i, 9), z(i, 2, 4), z(i, 2), z(i, 3)
    batch = B.DeviceBatch.empty(2, 5, "cpu")

    def bad(fn, *args, **kw):
        with pytest.raises((ValueError, TypeError)):
            fn(*args, **kw)

    bad(B.kv8_tables, refs, 16, two, two, table)                         # no batch and no rows
    bad(B.kv8_tables, refs, 16, two, three, table, batch)
    bad(B.kv8_tables, refs, 16, three, three, z(i, 3, 4), batch)         # a batch of two
    bad(B.kv8_tables, refs, 16, two, two, table, batch, 6)               # of five rows
    bad(B.kv8_tables, refs.long(), 16, two, two, table, batch)
    bad(B.kv8_tables, refs, 16, two, two, table.long(), batch)
    bad(B.kv8_tables, refs, 16, two, two, z(i, 4, 2).t(), batch)
    bad(B.kv8_tables, z(i, 18)[::2], 16, two, two, table, batch)
    bad(B.DeviceBatch, z(i, 3), two, z(i, 5), z(i, 5), z(i, 5), z(i, 1), 5)   # slots of 32 bits
    bad(B.DeviceBatch, z(i, 2), two, None, None, None, z(i, 1), 5)
    bad(B.DeviceBatch, z(i, 3), two, z(i, 4), None, None, z(i, 1), 5)
    bad(B.kv8_release, refs, table, three)
    bad(B.kv8_release, refs, table, None, z(torch.int64, 2))
    bad(B.kv8_reorder, refs, 16, table, two, three, z(i, 3, 5))          # another width
    bad(B.kv8_reorder, refs, 16, table, two, three, z(i, 2, 4))
    bad(B.kv8_reorder, refs, 16, table, three, three, z(i, 3, 4))
    bad(B.kv8_reorder, refs, 16, table, two, three, z(i, 3, 4), src=two)
    kv = B.DeviceKV8.empty(4, 2, 64, 16, "int8", "cpu")
    bad(B.kv8_copy_pages, [kv], three, two)
    bad(B.kv8_copy_pages, [kv], three, three, two)
    bad(B.beam_select, z(h, 6, 50), z(f, 6), 4)
    bad(B.beam_select, z(h, 6, 50), z(f, 6), 0)
    bad(B.beam_select, z(h, 6, 50), z(h, 6), 3)
    bad(B.beam_select, z(h, 6, 50), z(f, 5), 3)
    bad(B.beam_select, z(h, 50, 6).t(), z(f, 6), 3)
    bad(B.beam_select, z(torch.bfloat16, 6, 50), z(f, 6), 3)
    bad(B.beam_select, z(h, 6, 50), z(f, 6), 3, done=z(torch.bool, 6))
    bad(B.beam_select, z(h, 6, 50), z(f, 6), 3, norm=z(f, 3))
    bad(B.beam_select, z(h, 6, 50), z(f, 6), 3, parent=z(torch.int64, 6))
    q = z(h, 3, 256)
    bad(B.kv8_prefix_attention, kv, q, three, two, table, two, two, 4)
    bad(B.kv8_prefix_attention, kv, q.float(), three, two, table, two, z(i, 1), 4)
    bad(B.kv8_prefix_attention, kv, q, three, two, table, two.long(), z(i, 1), 4)
    bad(B.kv8_prefix_attention, kv, q[:, :200], three, two, table, two, z(i, 1), 4)
