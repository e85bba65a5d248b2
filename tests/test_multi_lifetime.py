"""Host-side tests of what a list's table keeps alive, with stand-in tensors
(no GPU)."""
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")

import zero_sharded_mixed_partition_amd as Z  # noqa: E402

from test_binding_checks import FakeDev  # noqa: E402
from test_multi_host import AL, BF16, fake_list  # noqa: E402


def moved(numels, at):
    return [FakeDev(n, BF16, AL + ((at + i) << 30)) for i, n in enumerate(numels)]


def test_a_recorded_table_keeps_its_gradients():
    """A replay reads the gradients that were described when the graph was
    recorded: they stay allocated after others are described, a table that no
    graph reads lets go of them."""
    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    t._captured = True                                     # as a call on a recording stream leaves it
    recorded = [weakref.ref(x) for x in g]
    for at in (8, 16):
        g = moved([100, 7], at)
        t.set_grads(g)
    later = [weakref.ref(x) for x in g]
    g = moved([100, 7], 24)
    t.set_grads(g)
    gc.collect()
    assert all(r() is not None for r in recorded)
    assert all(r() is None for r in later)                 # described after the recording, read by no graph
    assert t.grads == g


def test_other_streams_wait_for_the_tables_copy(monkeypatch):
    """The device copy is enqueued on the stream that was current when the table
    was built: any other one waits for it, once, before its first call reads it.
    A stream that records a graph cannot wait for work outside of it (the graph
    is recorded after a synchronization); its later, eager calls wait."""
    class Stream:
        device_index = 0

        def __init__(self, handle):
            self.cuda_stream, self.waited = handle, []

        def wait_event(self, e):
            self.waited.append(e)

    class Device:
        def record_stream(self, s):
            pass

        def data_ptr(self):
            return 1 << 45

    t = Z.TensorTable(*fake_list([100, 7]))
    copied = object()
    t._index, t.device, t._streams, t._ready = 0, Device(), {64}, copied
    recording = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: recording[0])
    own, other, third = Stream(64), Stream(128), Stream(192)
    for s in (own, other, other):
        t._ptrs(0, s)
    assert own.waited == [] and other.waited == [copied]
    current = Stream(256)
    monkeypatch.setattr(Z, "_raw_stream", lambda device: 256)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current)
    t._ptrs(0, None)
    t._ptrs(0, None)
    assert current.waited == [copied]
    recording[0] = True
    t._ptrs(0, third)
    assert third.waited == [] and t._captured
    recording[0] = False
    t._ptrs(0, third)
    assert third.waited == [copied]


def test_released_gradients():
    """A table lets go of its gradients when told to, and is not used until it
    has others; ones in the same place need no new description.  What a graph
    was recorded with stays."""
    m, a, b, g, p = fake_list([100, 7])
    t = Z.TensorTable(m, a, b, g, p)
    seen = [weakref.ref(x) for x in g]
    key, host = t._grad_key, t.host
    t.release_grads()
    t.release_grads()
    del g
    gc.collect()
    assert all(r() is None for r in seen)
    for call in (lambda: Z.zero_multi_adam_step(t, [Z.AdamHyper()], stream=0),
                 lambda: Z.zero_multi_unscale_norm_overflow(t, 1.0, FakeDev(1, torch.float64), FakeDev(1, torch.int32),
                                                            FakeDev(256, torch.uint8), stream=0)):
        with pytest.raises(ValueError, match="released"):
            call()
    g = fake_list([100, 7])[3]
    t.set_grads(g)                                         # where the former ones were
    assert t.grads == g and t._grad_key is key and t.host is host
    t._captured = True
    seen = [weakref.ref(x) for x in g]
    t.release_grads()
    del g
    gc.collect()
    assert all(r() is not None for r in seen)
    t.set_grads(moved([100, 7], 8))
    gc.collect()
    assert all(r() is not None for r in seen) and t.host is not host


def test_released_gradients_of_an_empty_list():
    t = Z.TensorTable.of_grads([])
    t.release_grads()
    t.set_grads([])
    assert t.grads == []
