"""GPU: MultiMuon with each type of updates and each adjustment of the learning rate
to a matrix's shape, against the models."""
import numpy as np
import pytest

import matmodel as M
import matspectra as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [(48, 80), (200, 40), (2, 40, 24), (130, 300), (300, 257), (1, 9)]
TYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


@pytest.mark.parametrize("device_state", [False, True])
@pytest.mark.parametrize("adjust", ["rms", "spectral", None])
@pytest.mark.parametrize("update", ["f16", "bf16"])
def test_two_steps(Z, update, adjust, device_state):
    """Momenta bit for bit; orthogonal updates within their bound of the definition
    on the rounded updates; masters bit for bit given those."""
    rng = np.random.default_rng(11)
    p = [(rng.normal(size=s) * 0.02).astype(np.float32) for s in SHAPES]
    gs = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in SHAPES]
    opt = Z.MultiMuon([torch.from_numpy(x).cuda() for x in p], gs, adjust=adjust, update_dtype=TYPE[update],
                      hyper=({"lr": 0.02, "weight_decay": 0.1},), device_state=device_state)
    m = [np.zeros(s, np.float32) for s in SHAPES]
    for step in range(2):
        for g in gs:
            g.copy_(torch.from_numpy(rng.normal(size=tuple(g.shape)) * 1e-2))
        assert opt.step() is (None if device_state else False)
        for k, shape in enumerate(SHAPES):
            m[k], u = M.momentum32(m[k], gs[k].cpu().float().numpy(), 1.0, 0.95, True)
            assert np.array_equal(opt.momentums[k].cpu().numpy().view(np.int32), m[k].view(np.int32)), (step, k)
            u = torch.from_numpy(u).to(TYPE[update]).double().numpy().reshape(-1, *shape[-2:])
            o = opt.updates[k].cpu()
            assert o.dtype == TYPE[update]
            for a, b in zip(u, o.double().numpy().reshape(u.shape)):
                ref, most = S.bound(a, update, M.COEFS)
                assert np.linalg.norm(b - ref) <= most < 0.2 * np.linalg.norm(ref), (step, k)
            rows, cols = shape[-2:]
            scale = {"rms": 0.2 * max(rows, cols) ** 0.5, "spectral": max(1.0, rows / cols) ** 0.5, None: 1.0}[adjust]
            p[k] = M.update32(p[k], o.float().numpy(), 0.02, scale, 0.1)
            assert np.array_equal(opt.masters[k].cpu().numpy().view(np.int32), p[k].view(np.int32)), (step, k)
    if device_state:
        assert opt.read_state().applied == 2
