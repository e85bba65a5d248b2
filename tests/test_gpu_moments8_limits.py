"""GPU: 8-bit moments at float32's upper end, against the oracle and the float32
model bit for bit; what is finite stays finite."""
import numpy as np
import pytest

import oracle.moments8 as O8
from f32model8 import adam8_update
from test_moments8_limits import FLT_MAX, HP, upper_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Z():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import zero_sharded_mixed_partition_amd as Z
    Z._L.lib()
    return Z


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pack_unpack(Z, m, v):
    n = m.numel()
    C = torch.empty(Z.zero_moments8_bytes(n), dtype=torch.uint8, device="cuda")
    S = torch.empty(Z.zero_scales8_bytes(n), dtype=torch.uint8, device="cuda")
    Z.zero_moments8_pack(C, S, m, v)
    M, V = torch.empty_like(m), torch.empty_like(v)
    Z.zero_moments8_unpack(M, V, C, S)
    return C.cpu().numpy(), S.cpu().numpy(), M.cpu().numpy(), V.cpu().numpy()


def test_the_largest_moments_pack_and_unpack(Z):
    m, v = (x.astype(np.float32) for x in upper_values())
    for k in (1, 5, m.size):
        for mm, vv in ((m[-k:], v[-k:]), (m[:k], v[:k])):
            C, S, M, V = pack_unpack(Z, cuda(mm), cuda(vv))
            want = O8.pack(mm, np.sqrt(vv).astype(np.float64) ** 2)
            assert np.array_equal(C, want[0]) and np.array_equal(S, want[1])
            dm, ds = O8.decode(*want, k)
            assert np.isfinite(M).all() and np.isfinite(V).all()
            assert np.array_equal(M, dm.astype(np.float32)) and np.array_equal(V, (ds * ds).astype(np.float32))
    # a NaN or inf beside them is still stored as NaN
    bad = cuda(np.array([FLT_MAX, np.inf, 1.0, np.nan], np.float32))
    C, S, M, V = pack_unpack(Z, bad, bad.clone())
    assert np.isnan(M[[1, 3]]).all() and np.isnan(V[[1, 3]]).all()


@pytest.mark.parametrize("n", [33, 256, 300])
@pytest.mark.parametrize("seed", [0, 1])
def test_the_largest_roots_are_stepped(Z, n, seed):
    """beta2 = 0 makes the root the gradient's magnitude; the next step, with an
    ordinary beta2, goes on from finite moments."""
    g = np.ldexp(np.linspace(200, 255.999, n), 56).astype(np.float32)
    p = np.linspace(-1, 1, n).astype(np.float32)
    c, s = np.zeros(8 * -(-n // 4), np.uint8), np.zeros(2 * -(-n // 32), np.uint8)
    P, C, S = cuda(p), cuda(c), cuda(s)
    table = Z.TensorTable([cuda(p)], [cuda(c)], [cuda(s)], [cuda(g)], state_bits=8)
    for step, over in ((1, {}), (2, dict(beta2=0.999)), (3, dict(beta2=0.999))):
        hp = dict(HP, step=step, **over)
        Z.zero_shard_adam8_step(P, C, S, cuda(g), None, Z.AdamHyper(**hp), seed=seed)
        Z.zero_multi_adam_step(table, [Z.AdamHyper(**hp)], seed=seed)
        p, c, s = adam8_update(p, c, s, g, 0.0, seed, **hp)
        for got in ((P, C, S), (table.masters[0], table.exp_avgs[0], table.exp_avg_sqs[0])):
            assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(got, (p, c, s))), step
        M, V = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        Z.zero_moments8_unpack(M, V, C, S)
        assert torch.isfinite(M).all() and torch.isfinite(V).all() and torch.isfinite(P).all()
