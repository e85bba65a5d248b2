"""Checkpoints of lists (no GPU): one of a longer list, or with other groups of
its tensors, is refused before anything is written."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

import zero_sharded_mixed_partition_amd as Z  # noqa: E402
from zero_sharded_mixed_partition_amd import checkpoint  # noqa: E402


@pytest.fixture(autouse=True)
def no_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(synchronize=lambda: None))


def opt(*sizes, groups, **kw):
    cols = [torch.full((n,), 1.0 + i) for i, n in enumerate(sizes)]
    return SimpleNamespace(state=None, t=0, scaler=Z.LossScaler(), hyper=[dict(lr=0.1), dict(lr=0.2)], seed=3, cols=cols,
                           groups=groups, checkpoint_arrays=lambda: {f"master_{i}": x for i, x in enumerate(cols)}, **kw)


def test_lists_of_other_tensors_or_groups_are_refused(tmp_path):
    saved = opt(5, 7, 9, groups=[0, 1, 0])
    for x in saved.cols:
        x.mul_(10)
    saved.t = 8
    checkpoint.save(saved, str(tmp_path))
    for other in (opt(5, 7, groups=[0, 1]), opt(5, 7, 9, groups=[0, 0, 1]), opt(5, 7, 9, 1, groups=[0, 1, 0, 0])):
        before = [x.clone() for x in other.cols]
        for load in (lambda: checkpoint.load(other, str(tmp_path)),
                     lambda: checkpoint.load_state_dict(other, checkpoint.state_dict(saved))):
            with pytest.raises((ValueError, FileNotFoundError)):
                load()
        assert other.t == 0 and all(torch.equal(x, y) for x, y in zip(before, other.cols))
    same = opt(5, 7, 9, groups=[0, 1, 0])
    checkpoint.load(same, str(tmp_path))
    assert same.t == 8 and all(torch.equal(x, y) for x, y in zip(saved.cols, same.cols))


def test_a_checkpoint_without_groups_still_loads():
    """Earlier checkpoints of lists do not hold them."""
    saved = checkpoint.state_dict(opt(5, 7, groups=[0, 1]))
    del saved["groups"]
    checkpoint.load_state_dict(opt(5, 7, groups=[0, 1]), saved)
