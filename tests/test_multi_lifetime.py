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
