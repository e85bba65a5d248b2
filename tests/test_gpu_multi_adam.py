"""GPU: whole steps of ShardAdam8 and MultiAdam: against their own calls and the
float32 model, host-scaled against device-resident state, recorded in a graph,
resumed from a checkpoint, over the fragments of a rank's shard, and with
gradients that move."""
import math

import numpy as np
import pytest

import oracle.moments8 as O8
from adam_bounds import adam64, assert_within
from f32model8 import adam8_update

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


def grads_for(n, step, scale, dtype=torch.float16, bad=False):
    rng = np.random.default_rng(1000 + step)
    g = torch.from_numpy((rng.normal(0, 1e-2, n) * scale).astype(np.float32)).to(dtype)
    if bad:
        g[n // 2] = float("inf")
    return g


def master_for(n):
    return torch.from_numpy(np.random.default_rng(1).normal(0, 0.02, n).astype(np.float32))


def same(a, b):
    return all(x.numel() == y.numel() and (not x.numel() or torch.equal(x.view(torch.uint8), y.view(torch.uint8)))
               for x, y in zip(a, b))


def arrays(opt):
    return list(opt.checkpoint_arrays().values())


# ---------------------------------------------------------------- ShardAdam8

def test_shard8_steps_follow_the_model(Z):
    """Five steps from zero moments, the third overflowing: master, codes and
    scales bit for bit, the copy its rounding, the scaler halved once."""
    n = 10_007
    opt = Z.ShardAdam8(master_for(n).cuda(), max_grad_norm=0.5, scaler=Z.LossScaler(scale=1024.0), seed=5, **HYPER)
    p = master_for(n).numpy()
    c, s = np.zeros(Z.zero_moments8_bytes(n), np.uint8), np.zeros(Z.zero_scales8_bytes(n), np.uint8)
    out = torch.zeros(n, dtype=torch.float16, device="cuda")
    t = 0
    for k in range(5):
        scale = opt.scaler.scale
        g = grads_for(n, k, scale, bad=k == 2)
        assert opt.step(g.cuda(), out) == (k == 2)
        if k != 2:
            t += 1
            p, c, s = adam8_update(p, c, s, g.float().numpy(), opt.sqnorm.item(), 5, step=t, inv_loss_scale=1.0 / scale,
                                   max_grad_norm=0.5, **HYPER)
        assert np.array_equal(opt.master.cpu().numpy(), p)
        assert np.array_equal(opt.moments8.cpu().numpy(), c) and np.array_equal(opt.scales8.cpu().numpy(), s)
        assert torch.equal(out.cpu(), torch.from_numpy(p).half())
    assert opt.t == 4 and opt.scaler.scale == 512.0
    m, v = opt.moments()
    dm, ds = O8.decode(c, s, n)
    assert np.array_equal(m.cpu().numpy(), dm.astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), (ds * ds).astype(np.float32))


def test_shard8_device_state_graph_and_accumulation(Z):
    """The host-scaled steps, the device-resident ones, recorded ones replayed
    between eager work, and ones whose gradient goes through the fp32 copy."""
    n = 30_011
    kw = dict(max_grad_norm=0.5, seed=9, **HYPER)
    mk = lambda **o: Z.ShardAdam8(master_for(n).cuda(), scaler=Z.LossScaler(scale=256.0, growth_interval=2), **kw, **o)  # noqa: E731
    host, dev, rec = mk(), mk(device_state=True), mk(device_state=True)
    outs = [torch.zeros(n, dtype=torch.float16, device="cuda") for _ in range(3)]
    G = torch.zeros(n, dtype=torch.float16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec.step(G, outs[2])
    for k in range(5):
        G.copy_(grads_for(n, k, host.scaler.scale, bad=k == 1))
        host.step(G, outs[0])
        dev.step(G, outs[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(arrays(host), arrays(dev)) and same(arrays(host), arrays(rec))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    st = dev.read_state()
    assert st.applied == host.t == 4 and dev.scaler.scale == host.scaler.scale and st.skipped == 1
    a, b = mk(), mk(device_state=True)
    acc = torch.empty(n, device="cuda")
    for opt in (a, b):
        for k in range(2):
            for j in range(3):
                opt.accumulate(acc, grads_for(n, 10 * k + j, 256.0).cuda(), first=j == 0, last=j == 2)
            opt.step(acc, None, norm_done=True)
    assert same(arrays(a), arrays(b))


@pytest.mark.parametrize("device_state", [False, True])
def test_shard8_resumes_bit_for_bit(Z, tmp_path, device_state):
    from zero_sharded_mixed_partition_amd import checkpoint
    n = 12_345
    mk = lambda seed: Z.ShardAdam8(master_for(n).cuda(), max_grad_norm=0.5, seed=seed, device_state=device_state,  # noqa: E731
                                   scaler=Z.LossScaler(scale=64.0), **HYPER)
    go = lambda o, ks: [o.step(grads_for(n, k, 64.0).cuda()) for k in ks]  # noqa: E731
    whole, first, second = mk(3), mk(3), mk(77)
    go(whole, range(6))
    go(first, range(3))
    checkpoint.save(first, str(tmp_path))
    checkpoint.load(second, str(tmp_path))
    assert second.seed == 3
    go(second, range(3, 6))
    assert same(arrays(whole), arrays(second))
    with pytest.raises(ValueError):
        d = checkpoint.state_dict(first)
        d["moments8"] = d["moments8"][:-1]
        checkpoint.load_state_dict(second, d)


def test_shard8_goes_on_from_fp32_moments(Z):
    n = 5000
    rng = np.random.default_rng(4)
    m, v = rng.normal(0, 1e-3, n).astype(np.float32), rng.uniform(1e-8, 1e-5, n).astype(np.float32)
    opt = Z.ShardAdam8.from_moments(master_for(n).cuda(), torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda(),
                                    applied_steps=7, **HYPER)
    a, b = (x.cpu().numpy().astype(np.float64) for x in opt.moments())
    _, s = O8.split(opt.moments8.cpu().numpy(), opt.scales8.cpu().numpy(), n)
    # half a code: 2^-4 of the value, or of the smallest normal code's spacing
    assert (np.abs(a - m) <= np.maximum(np.abs(m) * 2.0 ** -4, np.ldexp(1.0, s[0].astype(int) - 127 - 10))).all()
    root = np.sqrt(v.astype(np.float64))
    low = np.ldexp(1.0, s[1].astype(int) - 127 - 9)        # below it a root is raised to it
    assert (np.abs(np.sqrt(b) - root) <= np.maximum(root * (2.0 ** -4 + 2.0 ** -22), low)).all()
    assert opt.step(grads_for(n, 0, 1.0).cuda()) is False and opt.t == 8


# ---------------------------------------------------------------- MultiAdam

SIZES = [700, 5, 0, 8192, 20_001, 64]
GROUPS = [0, 1, 1, 0, 0, 1]
HYPERS = [dict(HYPER), dict(HYPER, weight_decay=0.0, lr=5e-4)]


def model_list(dtype=torch.float16, seed=0):
    rng = np.random.default_rng(seed)
    return ([torch.from_numpy(rng.normal(0, 0.02, n).astype(np.float32)) for n in SIZES],
            lambda k, scale, bad=False: [grads_for(n, 100 * k + i, scale, dtype, bad and i == 3) for i, n in enumerate(SIZES)])


def multi(Z, masters, grads, bits, **kw):
    out = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in SIZES]
    o = Z.MultiAdam([m.cuda() for m in masters], grads, out, hyper=HYPERS, groups=GROUPS, max_grad_norm=0.5,
                    state_bits=bits, scaler=Z.LossScaler(scale=512.0, growth_interval=2), seed=21, tensor_norms=True, **kw)
    return o, out


@pytest.mark.parametrize("bits", [32, 8])
def test_multi_steps_host_device_and_recorded(Z, bits):
    masters, make = model_list()
    G = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in SIZES]
    (host, o1), (dev, o2), (rec, o3) = (multi(Z, masters, G, bits, device_state=d) for d in (False, True, True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec.step()
    for k in range(4):
        scale = host.scaler.scale
        for t, g in zip(G, make(k, scale, bad=k == 1)):
            t.copy_(g)
        before = [x.clone() for x in arrays(host)]
        t0 = host.t
        assert host.step() == (k == 1)
        dev.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(arrays(host), arrays(dev)) and same(arrays(host), arrays(rec))
        assert same(o1, o2) and same(o1, o3)
        if k == 1:
            assert same(before, arrays(host))
            continue
        sums = [float((g.double() / scale).pow(2).sum()) for g in G]
        assert np.allclose(host.tensor_sqnorm.cpu().numpy(), sums, rtol=1e-13)
        assert math.isclose(host.sqnorm.item(), math.fsum(sums), rel_tol=1e-13)
        for i, n in enumerate(SIZES):
            hp = dict(HYPERS[GROUPS[i]], step=t0 + 1, inv_loss_scale=1.0 / scale, max_grad_norm=0.5)
            p0, a, b = (before[_at(what, i)].cpu().numpy() for what in ("master", "a", "b"))
            if bits == 8:
                m0, s0 = O8.decode(a, b, n)
                v0 = s0 * s0
            else:
                m0, v0 = a, b
            (p64, _, _), (dp, _, _) = adam64(p0, m0, v0, G[i].float().cpu().numpy(), host.sqnorm.item(), **hp)
            assert_within(f"step {k} tensor {i}", host.masters[i].cpu().numpy(), p64, dp)
            assert torch.equal(o1[i].cpu(), host.masters[i].cpu().half())
    st = dev.read_state()
    assert st.applied == host.t == 3 and dev.scaler.scale == host.scaler.scale


def _at(what, i):
    return {"master": 0, "a": 1, "b": 2}[what] * len(SIZES) + i


@pytest.mark.parametrize("bits", [32, 8])
def test_multi_with_moving_gradients_and_an_exchange(Z, bits):
    """New gradient tensors at every step, and an all-reduce hook that stands
    for three more ranks with the same gradients."""
    masters, make = model_list()
    G = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in SIZES]

    def exchange(sq, ovf):
        sq.mul_(4.0)

    runs = []
    for device_state in (False, True):
        for move in (False, True):
            opt, out = multi(Z, masters, G, bits, device_state=device_state)
            for k in range(3):
                g = [x.cuda() for x in make(k, 512.0)]
                if move:
                    opt.step(g, allreduce=exchange)
                else:
                    for t, x in zip(G, g):
                        t.copy_(x)
                    opt.step(allreduce=exchange)
            runs.append(arrays(opt) + out)
    assert all(same(runs[0], r) for r in runs[1:])
    # the scale doubled after the second clean step (growth_interval 2)
    sums = sum(float((x.double() / 1024.0).pow(2).sum()) for x in g)
    assert math.isclose(opt.sqnorm.item(), 4 * sums, rel_tol=1e-12)


@pytest.mark.parametrize("bits", [32, 8])
def test_multi_resumes_bit_for_bit(Z, tmp_path, bits):
    from zero_sharded_mixed_partition_amd import checkpoint
    masters, make = model_list(seed=3)
    G = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in SIZES]

    def go(o, ks):
        for k in ks:
            for t, x in zip(G, make(k, 512.0)):
                t.copy_(x)
            o.step()

    whole, first, second = (multi(Z, masters, G, bits, device_state=True)[0] for _ in range(3))
    go(whole, range(4))
    go(first, range(2))
    checkpoint.save(first, str(tmp_path))
    second.seed = 0
    checkpoint.load(second, str(tmp_path))
    go(second, range(2, 4))
    assert same(arrays(whole), arrays(second))


@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_of_several_dimensions(Z, tmp_path, bits):
    """Matrices, a scalar and an empty one: built from moments of their shapes,
    stepped as their flat forms are, saved and loaded."""
    from zero_sharded_mixed_partition_amd import checkpoint
    shapes = [(33, 7), (), (0, 4), (3, 5, 16), (1000,)]
    rng = np.random.default_rng(9)
    cols = [[torch.from_numpy(np.asarray(rng.uniform(1e-3, 1e-2, s), np.float32)).cuda() for s in shapes] for _ in range(3)]
    G = [torch.from_numpy(np.asarray(rng.normal(0, 1e-2, s), np.float32)).cuda() for s in shapes]
    opts = []
    for flat in (False, True, False):
        masters, m, v = ([(x.reshape(-1) if flat else x).clone() for x in col] for col in cols)
        opts.append(Z.MultiAdam(masters, [g.reshape(-1) if flat else g for g in G], hyper=[HYPER], moments=(m, v),
                                state_bits=bits))
    flat_arrays = lambda o: [x.reshape(-1) for x in arrays(o)]  # noqa: E731
    a, b, c = opts
    for o in (a, b):
        o.step()
    assert same(flat_arrays(a), flat_arrays(b))
    assert [tuple(x.shape) for x in a.masters] == shapes
    checkpoint.save(a, str(tmp_path))
    checkpoint.load(c, str(tmp_path))
    assert same(flat_arrays(a), flat_arrays(c))
    flat = checkpoint.state_dict(b)
    checkpoint.load_state_dict(c, flat)
    for o in (a, c):
        o.step()
    assert same(flat_arrays(a), flat_arrays(c))
    flat["hyper"] = flat["hyper"] * 2
    with pytest.raises(ValueError, match="groups"):
        checkpoint.load_state_dict(c, flat)


@pytest.mark.parametrize("bits", [32, 8])
def test_fragments_of_a_shard(Z, bits):
    """One rank's shard as a list of fragments that start anywhere.  With one
    group and no clipping its master, copy and (32 bits) moments equal the
    shard's own step bit for bit; the padding stays."""
    shapes, n_d, align = [(33, 7), (5,), (100, 13), (1,), (64,), (999,)], 3, 16
    _, S, _ = Z.zero_partition_plan(shapes, n_d, align)
    for rank in range(n_d):
        frags = Z.zero_rank_fragments(shapes, n_d, align, rank)
        rng = np.random.default_rng(rank)
        m, v = rng.normal(0, 1e-3, S).astype(np.float32), rng.uniform(1e-8, 1e-5, S).astype(np.float32)
        used = sum(f[3] for f in frags)
        p, g = master_for(S), grads_for(S, rank, 8.0, torch.bfloat16)
        p[used:] = 0
        g[used:] = 0
        P, G, O = p.cuda(), g.cuda(), torch.zeros(S, dtype=torch.bfloat16, device="cuda")
        M, V = torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda()
        opt = Z.MultiAdam.from_shard(frags, P, G, O, groups=[0] * len(shapes), moments=(M, V), hyper=[HYPER],
                                     state_bits=bits, scaler=Z.LossScaler.static(8.0), applied_steps=3)
        if bits == 32:
            Q, R = p.cuda(), torch.zeros(S, dtype=torch.bfloat16, device="cuda")
            shard = Z.ShardAdam(Q, M.clone(), V.clone(), scaler=Z.LossScaler.static(8.0), applied_steps=3, **HYPER)
            shard.step(G, R)
            opt.step()
            # the shard's step also takes its padding through the update, the list does not
            assert torch.equal(P[:used], Q[:used]) and torch.equal(O[:used], R[:used])
            for (_, _, b, n), x, y in zip(frags, opt.exp_avgs, opt.exp_avg_sqs):
                assert torch.equal(x, shard.exp_avg[b:b + n]) and torch.equal(y, shard.exp_avg_sq[b:b + n])
        else:
            start = [(a.cpu().numpy(), b.cpu().numpy()) for a, b in zip(opt.exp_avgs, opt.exp_avg_sqs)]
            opt.step()
            for i, (_, _, b, n) in enumerate(frags):
                want = adam8_update(p.numpy()[b:b + n], *start[i], g.float().numpy()[b:b + n], 0.0, 0, tensor=i, step=4,
                                    inv_loss_scale=1 / 8.0, max_grad_norm=0.0, **HYPER)
                assert np.array_equal(P[b:b + n].cpu().numpy(), want[0])
                assert np.array_equal(opt.exp_avgs[i].cpu().numpy(), want[1])
        assert not P[used:].any() and not O[used:].any()
