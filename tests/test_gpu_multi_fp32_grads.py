"""GPU: the fp32 gradient copy that a shard's accumulation forms (already
unscaled), stepped as a list: MultiAdam is told so with unscaled=True."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


@pytest.mark.parametrize("device_state", [False, True])
def test_an_accumulated_copy_is_stepped_as_a_list(Z, device_state):
    shapes, n_d, align, scale = [(33, 7), (5,), (100, 13), (64,)], 2, 16, 256.0
    _, S, _ = Z.zero_partition_plan(shapes, n_d, align)
    frags = Z.zero_rank_fragments(shapes, n_d, align, 0)
    used = sum(f[3] for f in frags)
    gen = torch.Generator().manual_seed(3)
    p = torch.zeros(S)
    p[:used] = torch.randn(used, generator=gen) * 0.02
    micro = []
    for _ in range(3):
        g = torch.zeros(S)
        g[:used] = torch.randn(used, generator=gen) * 1e-2 * scale
        micro.append(g.half().cuda())
    kw = dict(scaler=Z.LossScaler(scale=scale), device_state=device_state)
    shard = Z.ShardAdam(p.cuda(), torch.zeros(S, device="cuda"), torch.zeros(S, device="cuda"), **kw, **HYPER)
    acc = torch.empty(S, device="cuda")
    for j, g in enumerate(micro):
        shard.accumulate(acc, g, first=j == 0)
    master = p.cuda()
    kw["scaler"] = Z.LossScaler(scale=scale)
    opt = Z.MultiAdam.from_shard(frags, master, acc, groups=[0] * len(shapes), hyper=[HYPER], **kw)
    shard.step(acc)
    opt.step(unscaled=True)
    # without clipping the norm, whose squares the two passes add in another order, does not enter the update
    assert abs(opt.sqnorm.item() - shard.sqnorm.item()) <= 1e-13 * shard.sqnorm.item()
    assert torch.equal(master[:used], shard.master[:used])
    for (_, _, b, n), x, y in zip(frags, opt.exp_avgs, opt.exp_avg_sqs):
        assert torch.equal(x, shard.exp_avg[b:b + n]) and torch.equal(y, shard.exp_avg_sq[b:b + n])
