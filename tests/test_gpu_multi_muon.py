"""GPU: whole steps of MultiMuon: against the models, host-scaled against
device-resident state, recorded in a graph, resumed from a checkpoint, with
gradients that move, beside a MultiAdam of the other parameters, and empty."""
import math

import numpy as np
import pytest

import matmodel as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [(48, 80), (80, 48), (3, 40, 24), (130, 129), (300, 257)]
HYPER = ({"lr": 0.02, "momentum": 0.95, "weight_decay": 0.1}, {"lr": 0.01, "momentum": 0.9, "nesterov": False})
GROUPS = [0, 1, 0, 1, 0]


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def values(seed, size, shapes=SHAPES):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy((rng.normal(size=s) * size).astype(np.float32)) for s in shapes]


def grads(step, scale, bad=False):
    gs = [g.half() for g in values(100 + step, 1e-2 * scale)]
    if bad:
        gs[1][3, 5] = math.inf
    return [g.cuda() for g in gs]


def muon(Z, gs=None, **kw):
    gs = [torch.empty(s, dtype=torch.float16, device="cuda") for s in SHAPES] if gs is None else gs
    outs = [torch.empty(s, dtype=torch.float16, device="cuda") for s in SHAPES]
    kw = dict(dict(hyper=HYPER, groups=GROUPS, max_grad_norm=0.5, scaler=Z.LossScaler(scale=1024.0)), **kw)
    return Z.MultiMuon([p.cuda() for p in values(1, 0.02)], gs, outs, **kw), gs, outs


def state(opt):
    return [x.clone() for x in opt.checkpoint_arrays().values()]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8)) for x, y in zip(a, b))


def load(dst, src):
    for d, s in zip(dst, src):
        d.copy_(s)


def test_steps_follow_the_models(Z):
    """Four steps, the third overflowing: momenta bit for bit, orthogonal updates
    within their bound, masters bit for bit given those, copies their rounding,
    the scaler halved once."""
    opt, gs, outs = muon(Z, tensor_norms=True)
    p, m, scale, t = [x.numpy() for x in values(1, 0.02)], [np.zeros(s, np.float32) for s in SHAPES], 1024.0, 0
    for step in range(4):
        load(gs, grads(step, scale, bad=step == 2))
        assert opt.step() == (step == 2)
        if step == 2:
            scale /= 2
        else:
            t += 1
            sq = [float(np.sum((g.cpu().double().numpy() / scale) ** 2)) for g in gs]
            assert opt.sqnorm.item() == pytest.approx(sum(sq), rel=1e-12)
            assert opt.tensor_sqnorm.tolist() == pytest.approx(sq, rel=1e-12)
            factor = np.float32(1.0 / scale * min(1.0, 0.5 / (math.sqrt(opt.sqnorm.item()) + 1e-6)))
            for k, shape in enumerate(SHAPES):
                h = opt.hyper[GROUPS[k]]
                m[k], u = M.momentum32(m[k], gs[k].cpu().float().numpy(), factor, h["momentum"], h["nesterov"])
                u = torch.from_numpy(u).bfloat16().double().numpy().reshape(-1, *shape[-2:])
                o = opt.updates[k].cpu().double().numpy().reshape(u.shape)
                for a, b in zip(u, o):
                    ref, most = M.bound(a, "bf16")
                    assert np.linalg.norm(b - ref) <= most, (step, k)
                o = opt.updates[k].cpu().float().numpy()
                p[k] = M.update32(p[k], o, h["lr"], Z.muon_scale(shape, "rms"), h["weight_decay"])
        for k in range(len(SHAPES)):
            assert np.array_equal(opt.masters[k].cpu().numpy().view(np.int32), p[k].view(np.int32)), (step, k)
            assert np.array_equal(opt.momentums[k].cpu().numpy().view(np.int32), m[k].view(np.int32)), (step, k)
            assert torch.equal(outs[k].cpu(), torch.from_numpy(p[k]).half()), (step, k)
        assert opt.scaler.scale == scale and opt.t == t


@pytest.mark.parametrize("how", ["device", "exchange", "graph"])
def test_device_state_equals_host_scaled(Z, how):
    ref, rg, routs = muon(Z)
    opt, gs, outs = muon(Z, device_state=True)
    exchange = (lambda sq, ovf: None) if how == "exchange" else None
    graph = None
    if how == "graph":
        load(gs, grads(50, 1024.0))
        keep = state(opt)
        opt.step()                                     # kernels loaded before the recording
        load(opt.checkpoint_arrays().values(), keep)
        opt.state.tensor.copy_(Z.StepState(opt.scaler, 0, gs[0].device).tensor)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step()
    for step in range(6):
        new = grads(step, ref.scaler.scale, bad=step in (1, 4))
        load(rg, new)
        load(gs, new)
        assert ref.step() == (step in (1, 4))
        if graph is None:
            assert opt.step(allreduce=exchange) is None
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert same(state(ref), state(opt)) and same(routs, outs), step
    st = opt.read_state()
    assert (st.applied, st.skipped, opt.t) == (4, 2, 4) and opt.scaler.scale == ref.scaler.scale


@pytest.mark.parametrize("device_state", [False, True])
def test_checkpoints_resume(Z, tmp_path, device_state):
    a, ga, _ = muon(Z, device_state=device_state)
    for step in range(3):
        load(ga, grads(step, 1024.0 if step < 2 else 512.0, bad=step == 1))
        a.step()
    Z.checkpoint.save(a, str(tmp_path))
    b, gb, _ = muon(Z, device_state=device_state)
    Z.checkpoint.load(b, str(tmp_path))
    assert same(state(a), state(b)) and b.t == 2 and b.scaler.scale == 512.0
    for step in range(3, 5):
        for opt, g in ((a, ga), (b, gb)):
            load(g, grads(step, 512.0))
            opt.step()
    assert same(state(a), state(b))
    other, _, _ = muon(Z, groups=[0, 0, 0, 0, 0])
    with pytest.raises(ValueError, match="other groups"):
        Z.checkpoint.load(other, str(tmp_path))


def test_gradients_that_move_and_masters_of_their_own_kind(Z):
    """Gradients given anew each step, let go after it; the list goes on from given momenta."""
    a, ga, _ = muon(Z, momentums=[x.cuda() for x in values(7, 1e-2)])
    b, _, _ = muon(Z, momentums=[x.cuda() for x in values(7, 1e-2)])
    for step in range(3):
        new = grads(step, 1024.0)
        load(ga, new)
        a.step()
        b.step(new)
        b.release_grads()
        assert same(state(a), state(b)), step
    with pytest.raises(ValueError, match="released"):
        b.step()
    with pytest.raises(ValueError, match="shape"):
        b.step([g.reshape(-1) for g in new])
    with pytest.raises(ValueError, match="gradients for"):
        b.step(new[:-1])


def test_beside_a_list_of_the_other_parameters(Z):
    """Matrices by MultiMuon, vectors by MultiAdam, under one clip norm and one
    flag: both lists add the other's scalars, as ranks do."""
    vs = [torch.randn(k, device="cuda") for k in (48, 300)]
    vg = [torch.randn(k, device="cuda").half() for k in (48, 300)]
    opt, gs, _ = muon(Z)
    load(gs, grads(0, 1024.0))
    adam = Z.MultiAdam(vs, vg, max_grad_norm=0.5, scaler=Z.LossScaler(scale=1024.0))
    table = Z.TensorTable.of_grads(gs + vg)
    sq, ovf = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(Z.zero_multi_norm_workspace_bytes(table), dtype=torch.uint8, device="cuda")
    Z.zero_multi_unscale_norm_overflow(table, 1.0 / 1024, sq, ovf, ws)

    def both(s, o):
        s.copy_(sq)
        o.copy_(ovf)

    assert opt.step(allreduce=both) is False and adam.step(allreduce=both) is False
    assert opt.sqnorm.item() == adam.sqnorm.item() == sq.item()
    factor = np.float32(1.0 / 1024 * min(1.0, 0.5 / (math.sqrt(sq.item()) + 1e-6)))
    m, _ = M.momentum32(np.zeros(SHAPES[0], np.float32), gs[0].cpu().float().numpy(), factor, 0.95, True)
    assert np.array_equal(m.view(np.int32), opt.momentums[0].cpu().numpy().view(np.int32))


def test_an_empty_list_decides_with_the_others(Z):
    opt = Z.MultiMuon([], [], device="cuda", scaler=Z.LossScaler(scale=8.0))
    assert opt.step() is False and opt.t == 1
    assert opt.step(allreduce=lambda s, o: o.fill_(1)) is True and opt.scaler.scale == 4.0
    opt = Z.MultiMuon([], [], device="cuda", device_state=True)
    opt.step()
    assert opt.read_state().applied == 1
