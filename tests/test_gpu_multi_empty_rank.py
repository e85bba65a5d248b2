"""GPU: a rank whose shard is only padding takes part in the step: its norm is
zero, its scaler and step counter follow the exchanged scalars."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES, N_D, ALIGN = [(33, 7), (5,)], 4, 256
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def rank_of(Z, rank, bits, **kw):
    _, S, _ = Z.zero_partition_plan(SHAPES, N_D, ALIGN)
    gen = torch.Generator().manual_seed(rank)
    frags = Z.zero_rank_fragments(SHAPES, N_D, ALIGN, rank)
    used = sum(f[3] for f in frags)
    flat = [torch.zeros(S, device="cuda") for _ in range(2)]
    for x in flat:
        x[:used] = torch.randn(used, generator=gen).cuda() * 1e-2
    out = torch.zeros(S, dtype=torch.float16, device="cuda")
    return Z.MultiAdam.from_shard(frags, flat[0], flat[1].half(), out, groups=[0, 1], state_bits=bits,
                                  hyper=[HYPER, dict(HYPER, weight_decay=0.0)], max_grad_norm=0.5, tensor_norms=True,
                                  scaler=Z.LossScaler(scale=64.0, growth_interval=2), **kw)


@pytest.mark.parametrize("bits", [32, 8])
def test_an_empty_rank_follows_the_others(Z, bits, tmp_path):
    from zero_sharded_mixed_partition_amd import checkpoint
    for device_state in (False, True):
        full, empty = (rank_of(Z, r, bits, device_state=device_state) for r in (0, 2))
        assert full.table.n_tensors == 2 and empty.table.n_tensors == 0
        for k in range(5):
            if k == 1:
                full.table.grads[0][3] = float("inf")
            elif k == 2:
                full.table.grads[0][3] = 0.0
            seen = {}

            def exchange(sq, ovf):                         # the other ranks' scalars: this one's only are not zero
                seen["own"] = sq.clone(), ovf.clone()

            def received(sq, ovf):
                assert sq.item() == 0.0 and ovf.item() == 0
                sq.copy_(seen["own"][0]), ovf.copy_(seen["own"][1])

            skipped = full.step(allreduce=exchange), empty.step([], allreduce=received)
            assert skipped == ((None, None) if device_state else (k == 1, k == 1))
        if device_state:
            full.read_state(), empty.read_state()
        # 64 at first, halved by the second step, doubled after two clean ones (the fourth); the fifth is clean
        assert empty.t == full.t == 4 and empty.scaler.scale == full.scaler.scale == 64.0
        checkpoint.save(empty, str(tmp_path / str(device_state)))
        again = rank_of(Z, 2, bits, device_state=device_state)
        checkpoint.load(again, str(tmp_path / str(device_state)))
        assert again.t == 4 and again.scaler.scale == 64.0


@pytest.mark.parametrize("bits", [32, 8])
def test_an_empty_rank_alone_and_recorded(Z, bits):
    eager, rec, host = (rank_of(Z, 3, bits, device_state=d) for d in (True, True, False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec.step()
    for _ in range(3):
        eager.step()
        assert host.step() is False
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    for opt in (eager, rec):
        assert opt.read_state().applied == host.t == 3 and opt.scaler.scale == host.scaler.scale == 128.0
        assert opt.sqnorm.item() == 0.0
