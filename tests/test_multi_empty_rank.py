"""A rank whose shard is only padding holds no fragment: its MultiAdam is an
empty list (no GPU; the buffers are host ones)."""
import pytest

torch = pytest.importorskip("torch")

import zero_sharded_mixed_partition_amd as Z  # noqa: E402


@pytest.fixture
def host_buffers(monkeypatch):
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, pin_memory=False, **kw: empty(*a, **kw))
    monkeypatch.setattr(torch.cuda, "Event", lambda: None)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_rank_without_fragments(host_buffers, bits):
    shapes = [(33, 7), (5,)]
    _, S, _ = Z.zero_partition_plan(shapes, 4, 256)
    for rank in (1, 2, 3):
        frags = Z.zero_rank_fragments(shapes, 4, 256, rank)
        assert frags == []
        master, grad, out = torch.zeros(S), torch.zeros(S).half(), torch.zeros(S).half()
        opt = Z.MultiAdam.from_shard(frags, master, grad, out, groups=[0, 1], moments=(master, master),
                                     hyper=[{}, dict(weight_decay=0.0)], state_bits=bits, tensor_norms=True)
        assert opt.table.n_tensors == 0 and opt.checkpoint_arrays() == {} and opt.masters == opt.exp_avgs == []
        assert opt.workspace.numel() == 256 and opt.tensor_sqnorm.numel() == 0
        opt.table.set_grads([])
    assert Z.MultiAdam([], [], device="cpu").table.n_tensors == 0
